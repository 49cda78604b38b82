"""Host-side tests of the four-bit operators' C ABI (no GPU needed): every
declared entry point is exported, and each invalid argument is rejected with its
documented status before the HIP runtime is touched. Every call here is invalid
or empty, so nothing is launched; the fake device pointers are never read.
"""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, DTYPE, VALUE, UNSUP, HIP, ALIGN = range(8)
A, A2, A3 = 0x10000, 0x20000, 0x30000

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="host-only validation tests (fake device pointers)")


@pytest.fixture(scope="module")
def lib():
    import prompt_conditioned_keypoint_amd as gkd
    return gkd.load()


def heads(data=A, batch=4096, token=512, head=64):
    from prompt_conditioned_keypoint_amd.binding import GkdHeads
    return ctypes.byref(GkdHeads(data, batch, token, head))


def cache(codes=A2, scales=A3, pages=9, page=64, Hk=2, D=64):
    from prompt_conditioned_keypoint_amd.binding import GkdCache
    return ctypes.byref(GkdCache(codes, scales, pages, page, Hk, D))


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "gkdfp4.h")).read()
    names = set(re.findall(r"^GKD_API \w+ (gkd_\w+)\(", text, re.M))
    assert names == {"gkd_fp4_version", "gkd_quantize_fp4", "gkd_linear_fp4_workspace_size",
                     "gkd_linear_fp4", "gkd_cache_append", "gkd_cache_read",
                     "gkd_cache_attention_workspace_size", "gkd_cache_attention"}
    for n in names:
        assert hasattr(lib, n), n
    assert lib.gkd_fp4_version() == 1


def quant(lib, x=A, ldx=64, N=4, K=64, dtype=1, flags=0, codes=A2, scales=A3):
    return lib.gkd_quantize_fp4(x, ldx, N, K, dtype, flags, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), UNSUP), (dict(dtype=2), DTYPE), (dict(N=-1), SHAPE), (dict(K=0), SHAPE),
    (dict(ldx=63), SHAPE), (dict(K=48), UNSUP), (dict(x=None), NULL), (dict(codes=None), NULL),
    (dict(scales=None), NULL), (dict(codes=A2 + 8), ALIGN), (dict(scales=A3 + 4), ALIGN),
    (dict(x=A + 8), ALIGN), (dict(ldx=68), ALIGN), (dict(ldx=66, dtype=0), ALIGN),
])
def test_quantize_rejects(lib, kw, status):
    assert quant(lib, **kw) == status
    assert lib.gkd_last_error().decode() != ""


def lin(lib, x=A, ldx=64, codes=A2, scales=A3, bias=None, res=None, ldr=0, M=4, N=32, K=64, act=0,
        out_dtype=1, flags=0, out=A3, ldo=32, ws=A, ws_bytes=1 << 40):
    return lib.gkd_linear_fp4(x, ldx, codes, scales, bias, res, ldr, M, N, K, act, out_dtype, flags,
                              out, ldo, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), UNSUP), (dict(out_dtype=-1), DTYPE), (dict(act=5), VALUE), (dict(act=-1), VALUE),
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=0), SHAPE), (dict(M=1 << 26), SHAPE),
    (dict(N=1 << 25, ldo=1 << 25), SHAPE), (dict(M=1 << 16, N=1 << 15, ldo=1 << 15), SHAPE),
    (dict(K=1 << 22, ldx=1 << 22), SHAPE), (dict(ldx=1 << 22), SHAPE), (dict(ldx=0), SHAPE),
    (dict(ldx=63), SHAPE), (dict(K=48), UNSUP), (dict(ldo=31), SHAPE), (dict(res=A, ldr=31), SHAPE),
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL),
    (dict(x=A + 8), ALIGN), (dict(ldx=68), ALIGN), (dict(codes=A2 + 8), ALIGN),
    (dict(scales=A3 + 1), ALIGN), (dict(bias=A + 1), ALIGN), (dict(out=A + 2, out_dtype=0), ALIGN),
    (dict(res=A + 2, ldr=32, out_dtype=0), ALIGN),
])
def test_linear_rejects(lib, kw, status):
    assert lin(lib, **kw) == status
    assert lib.gkd_last_error().decode() != ""


def test_linear_empty_is_ok(lib):
    assert lin(lib, M=0, x=None, out=None) == OK
    assert lin(lib, N=0, codes=None, scales=None, out=None, ldo=0) == OK
    size = lib.gkd_linear_fp4_workspace_size
    assert size(0, 8, 64) == 0 and size(8, 0, 64) == 0 and size(-1, 8, 64) == 0 and size(8, 8, 48) == 0


def append(lib, k=None, v=None, B=2, T=3, start=None, count=None, c=None, table=A, L=4, dtype=1, flags=0):
    return lib.gkd_cache_append(k or heads(), v or heads(), B, T, start, count, c or cache(), table, L,
                                dtype, flags, None)


def read(lib, c=None, table=A, L=4, B=2, T=3, start=None, count=None, flags=0, k=None, v=None):
    return lib.gkd_cache_read(c or cache(), table, L, B, T, start, count, flags, k or heads(),
                              v or heads(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), UNSUP), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(B=1 << 16, T=1 << 15), SHAPE),
    (dict(L=-1), SHAPE), (dict(L=1 << 24), SHAPE), (dict(table=None), NULL), (dict(table=A + 2), ALIGN),
    (dict(start=A + 1), ALIGN), (dict(count=A + 2), ALIGN),
])
def test_append_and_read_reject(lib, kw, status):
    for call in (append, read):
        assert call(lib, **kw) == status
        assert lib.gkd_last_error().decode() != ""


def test_append_and_read_reject_tokens_that_32_bits_do_not_count(lib):
    for call in (append, read):
        assert call(lib, B=1, T=1 << 30) == SHAPE and call(lib, B=1, T=(1 << 31) - 1) == SHAPE
        assert call(lib, B=0, T=(1 << 30) - 1) == 0


BAD_CACHES = [(dict(pages=-1), SHAPE), (dict(page=0), SHAPE), (dict(page=1 << 17), SHAPE), (dict(Hk=0), SHAPE),
              (dict(Hk=1 << 17), SHAPE), (dict(D=0), SHAPE), (dict(D=96), UNSUP), (dict(page=48), UNSUP),
              (dict(page=16), UNSUP), (dict(codes=None), NULL), (dict(scales=None), NULL),
              (dict(codes=A + 8), ALIGN), (dict(scales=A + 2), ALIGN)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_cache_call_checks_the_cache(lib, kw, status):
    for call in (append, read, attn):
        assert call(lib, c=cache(**kw)) == status, call
        assert lib.gkd_last_error().decode() != ""


def test_append_and_read_check_heads(lib):
    assert append(lib, dtype=2) == DTYPE
    for name in ("k", "v"):
        for kw, status in ((dict(data=None), NULL), (dict(data=A + 8), ALIGN), (dict(token=516), ALIGN),
                           (dict(head=-64), SHAPE)):
            assert append(lib, **{name: heads(**kw)}) == status
            assert read(lib, **{name: heads(**kw)}) == status
        for kw in (dict(batch=0), dict(token=0), dict(head=0)):
            assert read(lib, **{name: heads(**kw)}) == SHAPE              # an output's places are its own
            assert append(lib, **{name: heads(**kw)}, start=A + 1) == ALIGN
    assert append(lib, k=heads(token=514), dtype=0) == ALIGN
    for call in (append, read):
        assert call(lib, B=0) == OK and call(lib, T=0, table=None) == OK
    # without pages or columns there is no place: nothing is launched
    assert append(lib, c=cache(pages=0, codes=None, scales=None)) == OK
    assert append(lib, L=0, table=None) == OK


def attn(lib, q=None, c=None, table=A, L=4, length=None, q_len=None, B=2, Tq=3, Hq=4, scale=0.125, flags=0,
         out=None, ws=A, ws_bytes=1 << 40):
    return lib.gkd_cache_attention(q or heads(), c or cache(), table, L, length, q_len, B, Tq, Hq, scale,
                                   flags, out or heads(A3), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=2), UNSUP), (dict(B=-1), SHAPE), (dict(Tq=-1), SHAPE), (dict(Hq=0), SHAPE),
    (dict(B=1 << 16, Tq=1 << 14), SHAPE), (dict(B=1 << 20, Tq=1), SHAPE), (dict(B=1 << 16, Tq=256), SHAPE),
    (dict(Hq=3), UNSUP), (dict(L=-1), SHAPE), (dict(L=1 << 24), SHAPE),
    (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=float("inf")), VALUE),
    (dict(scale=float("nan")), VALUE), (dict(scale=3e38), VALUE),
    (dict(table=None), NULL), (dict(table=A + 2), ALIGN), (dict(length=A + 2), ALIGN), (dict(q_len=A + 1), ALIGN),
])
def test_attention_rejects(lib, kw, status):
    assert attn(lib, **kw) == status
    assert lib.gkd_last_error().decode() != ""


def test_attention_rejects_operands(lib):
    for name in ("q", "out"):
        assert attn(lib, **{name: heads(data=None)}) == NULL, name
        assert attn(lib, **{name: heads(data=A + 8)}) == ALIGN, name
        assert attn(lib, **{name: heads(token=516)}) == ALIGN, name
        assert attn(lib, **{name: heads(head=-64)}) == SHAPE, name
    for kw in (dict(batch=0), dict(token=0), dict(head=0)):
        assert attn(lib, out=heads(**kw)) == SHAPE
        assert attn(lib, q=heads(**kw), length=A + 2) == ALIGN
    assert attn(lib, B=0) == OK and attn(lib, Tq=0, ws=None) == OK


def test_attention_checks_its_workspace(lib):
    size = lib.gkd_cache_attention_workspace_size
    need = size(1, 1, 8, 2, 64, 64, 256)
    assert need > 0
    kw = dict(B=1, Tq=1, Hq=8, L=256)
    assert attn(lib, ws=None, **kw) == NULL
    assert attn(lib, ws=A + 64, **kw) == ALIGN
    assert attn(lib, ws_bytes=need - 1, **kw) == VALUE
    for bad in ((0, 1, 8, 2, 64, 64, 256), (1, 0, 8, 2, 64, 64, 256), (1, 1, 7, 2, 64, 64, 256),
                (1, 1, 8, 2, 96, 64, 256), (1, 1, 8, 2, 64, 48, 256), (1, 1, 8, 0, 64, 64, 256),
                (1, 1, 8, 2, 64, 64, -1), (1, 1, 8, 2, 64, 65536, 1 << 20)):
        assert size(*bad) == 0, bad


def test_attention_shares_what_one_long_sequence_would_hold_up(lib):
    """Work is cut evenly, which takes a workspace, wherever the room lets one tile outlast
    many others, or the key heads leave XCDs without work."""
    size = lib.gkd_cache_attention_workspace_size
    for B, Tq, Hq, Hk, D, room in ((512, 1, 32, 8, 128, 262144), (512, 1, 32, 8, 128, 32768),
                                   (600, 1, 16, 8, 128, 65536),
                                   (1, 4096, 32, 4, 128, 16384), (1, 4096, 24, 12, 128, 16384)):
        assert size(B, Tq, Hq, Hk, D, 64, room // 64) > 0, (B, Tq, Hq, Hk, D, room)
    for B, Tq, Hq, Hk, D, room in ((512, 1, 32, 8, 128, 16384), (1, 4096, 32, 8, 128, 65536),
                                   (256, 64, 16, 16, 64, 32768)):
        assert size(B, Tq, Hq, Hk, D, 64, room // 64) == 0, (B, Tq, Hq, Hk, D, room)


def test_attention_shares_the_work_of_any_number_of_sequences(lib):
    size = lib.gkd_cache_attention_workspace_size
    for B in (1024, 1025, 2049, 8192):
        assert size(B, 1, 8, 1, 128, 64, 4096) > 0, B


def test_python_calls_reject_cpu_tensors():
    import prompt_conditioned_keypoint_amd as gkd
    bf, u8 = torch.bfloat16, torch.uint8
    x, h = torch.zeros(2, 64, dtype=bf), torch.zeros(1, 2, 2, 64, dtype=bf)
    wc, ws = torch.zeros(3, 32, dtype=u8), torch.zeros(3, 2, dtype=u8)
    cc, cs = torch.zeros(4, 2, 2, 32, 32, dtype=u8), torch.zeros(4, 2, 2, 32, 2, dtype=u8)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: gkd.quantize_fp4(x), lambda: gkd.linear_fp4(x, wc, ws),
                 lambda: gkd.cache_append(h, h, cc, cs, table), lambda: gkd.cache_read(cc, cs, table, 3),
                 lambda: gkd.cache_attention(h, cc, cs, table)):
        with pytest.raises(ValueError):
            call()


def test_python_calls_refuse_sizes_past_32_bits():
    import prompt_conditioned_keypoint_amd as gkd
    for bad in (2**31, 2**32, 2**32 + 5):
        for call, n in ((gkd.linear_fp4_workspace_size, 3), (gkd.cache_attention_workspace_size, 7)):
            for i in range(n):
                with pytest.raises(gkd.GkdError) as e:
                    call(*(bad if j == i else 64 for j in range(n)))
                assert e.value.status == SHAPE
