"""Host-side tests of the token operators' C ABI (no GPU needed): every
declared entry point is exported, and each invalid argument is rejected with
its documented status before the HIP runtime is touched. Every call here is
invalid or empty, so nothing is launched; the fake device pointers are never
read.
"""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, DTYPE, VALUE, UNSUP, HIP, ALIGN = range(8)
A, A2, A3, MIS = 0x10000, 0x20000, 0x30000, 0x10002

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="host-only validation tests (fake device pointers)")


@pytest.fixture(scope="module")
def lib():
    import prompt_conditioned_keypoint_amd as gkd
    return gkd.load()


def heads(data=A, batch=4096, token=512, head=64):
    from prompt_conditioned_keypoint_amd.binding import GkdHeads
    return ctypes.byref(GkdHeads(data, batch, token, head))


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "gkdtokens.h")).read()
    names = set(re.findall(r"^GKD_API \w+ (gkd_\w+)\(", text, re.M))
    assert names == {"gkd_tokens_version", "gkd_linear_workspace_size", "gkd_linear",
                     "gkd_qk_norm_rope", "gkd_prefix_attention_workspace_size",
                     "gkd_prefix_attention"}
    for n in names:
        assert hasattr(lib, n), n
    assert lib.gkd_tokens_version() == 1


def lin(lib, x=A, ldx=64, w=A2, ldw=64, bias=None, res=None, ldr=0, M=4, N=32, K=64, act=0, dtype=1,
        out_dtype=1, flags=0, out=A3, ldo=32, ws=None, ws_bytes=0):
    return lib.gkd_linear(x, ldx, w, ldw, bias, res, ldr, M, N, K, act, dtype, out_dtype, flags, out,
                          ldo, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), UNSUP),
    (dict(dtype=2), DTYPE),
    (dict(out_dtype=-1), DTYPE),
    (dict(dtype=0), UNSUP),
    (dict(act=5), VALUE),
    (dict(act=-1), VALUE),
    (dict(M=-1), SHAPE),
    (dict(N=-1), SHAPE),
    (dict(K=0), SHAPE),
    (dict(M=1 << 26), SHAPE),
    (dict(N=1 << 25, ldo=1 << 25), SHAPE),
    (dict(M=1 << 18, N=1 << 18, ldo=1 << 18), SHAPE),      # M N >= 2^36
    (dict(ldx=63), SHAPE),
    (dict(ldw=0), SHAPE),                     # rows that repeat
    (dict(ldx=1 << 22), SHAPE),
    (dict(ldo=31), SHAPE),
    (dict(res=A, ldr=31), SHAPE),
    (dict(x=None), NULL),
    (dict(w=None), NULL),
    (dict(out=None), NULL),
    (dict(x=A + 8), ALIGN),
    (dict(w=A + 2), ALIGN),
    (dict(bias=A + 1), ALIGN),
    (dict(out=A + 2, out_dtype=0), ALIGN),
    (dict(res=A + 2, ldr=32, out_dtype=0), ALIGN),
    (dict(K=63), NULL),                       # rows to copy, no workspace
    (dict(ldx=65), NULL),
    (dict(K=63, ws=A + 16, ws_bytes=1 << 30), ALIGN),
    (dict(K=63, ws=A, ws_bytes=100), VALUE),
])
def test_linear_rejects(lib, kw, status):
    assert lin(lib, **kw) == status
    assert lib.gkd_last_error().decode() != ""


def test_linear_empty_is_ok_and_workspace_follows_the_rows(lib):
    assert lin(lib, M=0, x=None, out=None) == OK
    assert lin(lib, N=0, w=None, out=None, ldo=0) == OK
    size = lib.gkd_linear_workspace_size
    assert size(4, 32, 64, 64, 64) == 0
    assert size(4, 32, 64, 72, 80) == 0
    assert size(4, 32, 64, 65, 64) == 512                   # x: 4 rows of 128 bytes
    assert size(4, 32, 63, 64, 64) == 512 + 4096            # both
    assert size(-1, 32, 63, 64, 64) == 0


def rope(lib, q=None, Hq=4, k=None, Hk=2, B=2, T=3, D=64, pos=A, pos_batch=0, n_axes=2, freqs=A2,
         rot=64, wq=None, wk=None, eps=1e-6, dtype=1, flags=0, qo=None, ko=None, no_k=False):
    k_, ko_ = (None, None) if no_k else (k or heads(), ko or heads(A3))
    return lib.gkd_qk_norm_rope(q or heads(), Hq, k_, Hk, B, T, D, pos, pos_batch, n_axes, freqs, rot,
                                wq, wk, eps, dtype, flags, qo or heads(A2), ko_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=2), UNSUP),
    (dict(dtype=3), DTYPE),
    (dict(B=-1), SHAPE),
    (dict(T=-1), SHAPE),
    (dict(Hq=0), SHAPE),
    (dict(Hk=-1), SHAPE),
    (dict(D=0, rot=0), SHAPE),
    (dict(rot=0), SHAPE),
    (dict(rot=7), SHAPE),
    (dict(rot=66), SHAPE),
    (dict(n_axes=0), SHAPE),
    (dict(pos_batch=-1), SHAPE),
    (dict(D=514, rot=64), UNSUP),
    (dict(n_axes=9), UNSUP),
    (dict(Hq=70000), UNSUP),
    (dict(eps=-1.0), VALUE),
    (dict(eps=float("nan")), VALUE),
    (dict(no_k=True), NULL),                  # Hk without keys
    (dict(Hk=0), NULL),                       # keys without Hk
    (dict(pos=None), NULL),
    (dict(freqs=None), NULL),
    (dict(pos=A + 2), ALIGN),
    (dict(wq=A + 1), ALIGN),
    (dict(wk=A + 2, dtype=0), ALIGN),
])
def test_rope_rejects(lib, kw, status):
    assert rope(lib, **kw) == status
    assert lib.gkd_last_error().decode() != ""


def test_rope_rejects_operands(lib):
    assert rope(lib, q=heads(data=None)) == NULL
    assert rope(lib, ko=heads(data=None)) == NULL
    assert rope(lib, k=heads(token=-8)) == SHAPE
    assert rope(lib, qo=heads(data=A + 1)) == ALIGN
    assert rope(lib, q=heads(data=A + 2), dtype=0) == ALIGN
    # an output's elements have places of their own, an input's need not
    for kw in (dict(batch=0), dict(token=0), dict(head=0)):
        assert rope(lib, qo=heads(**kw)) == SHAPE and rope(lib, ko=heads(**kw)) == SHAPE
        assert rope(lib, q=heads(**kw), freqs=None) == NULL
    assert rope(lib, qo=heads(batch=0), B=1, freqs=None) == NULL
    assert rope(lib, B=0) == OK and rope(lib, T=0, Hk=0, no_k=True) == OK


def attn(lib, q=None, kp=None, vp=None, P=16, ko=None, vo=None, S=8, own_len=None, q_len=None,
         mask=None, B=2, Tq=3, Hq=4, Hk=2, D=64, scale=0.125, dtype=1, flags=0, out=None, ws=A,
         ws_bytes=1 << 40):
    return lib.gkd_prefix_attention(q or heads(), kp or heads(), vp or heads(), P, ko or heads(),
                                    vo or heads(), S, own_len, q_len, mask, B, Tq, Hq, Hk, D, scale,
                                    dtype, flags, out or heads(A3), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=2), UNSUP),
    (dict(dtype=2), DTYPE),
    (dict(dtype=0), UNSUP),
    (dict(B=-1), SHAPE),
    (dict(Tq=-1), SHAPE),
    (dict(Hk=0), SHAPE),
    (dict(Hq=0), SHAPE),
    (dict(P=-1), SHAPE),
    (dict(S=1 << 30), SHAPE),
    (dict(D=0), SHAPE),
    (dict(B=1 << 16, Tq=1 << 14), SHAPE),      # B Tq Hq >= 2^31
    (dict(B=1 << 22, Tq=1), SHAPE),            # 2^23 groups of heads
    (dict(B=1 << 14, Tq=16448, Hk=4), SHAPE),  # 129 tiles of each of 2^16
    (dict(D=96), UNSUP),
    (dict(Hk=3), UNSUP),
    (dict(scale=0.0), VALUE),
    (dict(scale=-1.0), VALUE),
    (dict(scale=float("inf")), VALUE),
    (dict(scale=3e38, own_len=A + 2), VALUE),  # times log2(e) past float32
    (dict(own_len=A + 2), ALIGN),
    (dict(q_len=A + 1), ALIGN),
])
def test_attention_rejects(lib, kw, status):
    assert attn(lib, **kw) == status
    assert lib.gkd_last_error().decode() != ""


def test_attention_rejects_operands(lib):
    for name in ("q", "kp", "vp", "ko", "vo", "out"):
        assert attn(lib, **{name: heads(data=None)}) == NULL, name
        assert attn(lib, **{name: heads(data=A + 8)}) == ALIGN, name
        assert attn(lib, **{name: heads(token=516)}) == ALIGN, name
        assert attn(lib, **{name: heads(head=-64)}) == SHAPE, name
    for name in ("kp", "vp", "ko", "vo"):
        assert attn(lib, **{name: heads(token=1 << 25)}) == SHAPE, name
    for kw in (dict(batch=0), dict(token=0), dict(head=0)):
        assert attn(lib, out=heads(**kw)) == SHAPE
        assert attn(lib, q=heads(**kw), ko=heads(**kw), own_len=A + 2) == ALIGN
    assert attn(lib, out=heads(head=0, token=64), Hq=1, Hk=1, own_len=A + 2) == ALIGN
    assert attn(lib, B=0) == OK and attn(lib, Tq=0, ws=None) == OK


def test_attention_checks_its_workspace(lib):
    size = lib.gkd_prefix_attention_workspace_size
    need = size(48, 1, 32, 8, 128, 32768, 1024)
    assert need > 0
    kw = dict(B=48, Tq=1, Hq=32, Hk=8, D=128, P=32768, S=1024)
    assert attn(lib, ws=None, **kw) == NULL
    assert attn(lib, ws=A + 64, **kw) == ALIGN
    assert attn(lib, ws_bytes=need - 1, **kw) == VALUE
    assert size(0, 1, 32, 8, 128, 10, 10) == 0 and size(1, 1, 32, 7, 128, 10, 10) == 0


def test_python_calls_reject_cpu_tensors_and_bad_shapes():
    import prompt_conditioned_keypoint_amd as gkd
    bf = torch.bfloat16
    x, w = torch.zeros(2, 8, dtype=bf), torch.zeros(3, 8, dtype=bf)
    with pytest.raises(ValueError):
        gkd.linear(x, w)
    h = torch.zeros(1, 2, 2, 64, dtype=bf)
    with pytest.raises(ValueError):
        gkd.qk_norm_rope(h, h, torch.zeros(2, 1), torch.zeros(1, 32))
    with pytest.raises(ValueError):
        gkd.prefix_attention(h, h[0], h[0])


def test_python_calls_refuse_sizes_past_32_bits():
    """The C ABI's sizes are ints; a larger one must not arrive cut short."""
    import prompt_conditioned_keypoint_amd as gkd
    from prompt_conditioned_keypoint_amd.binding import _int_sizes
    _int_sizes("f", 0, 5, 2**31 - 1)
    for bad in (2**31, 2**32, 2**32 + 5, 2**63):
        with pytest.raises(gkd.GkdError) as e:
            _int_sizes("f", 1, bad, 2)
        assert e.value.status == SHAPE
        for i in range(3):
            with pytest.raises(gkd.GkdError) as e:
                gkd.linear_workspace_size(*(bad if j == i else 8 for j in range(3)))
            assert e.value.status == SHAPE
        for i in range(7):
            with pytest.raises(gkd.GkdError) as e:
                gkd.prefix_attention_workspace_size(*(bad if j == i else 8 for j in range(7)))
            assert e.value.status == SHAPE
    assert gkd.linear_workspace_size(2**31 - 1, 8, 8) == 0      # past the call's own limits: it takes none


def test_row_stride_takes_evenly_spaced_rows_only():
    from prompt_conditioned_keypoint_amd.binding import _row_stride
    t = torch.zeros(4, 6, 16)
    assert _row_stride(t, "t") == 16
    assert _row_stride(t[:, :, :8], "t") == 16
    assert _row_stride(t[:, ::2, :8], "t") == 32
    assert _row_stride(t[:, 0], "t") == 96
    assert _row_stride(t[0, 0], "t") == 16
    assert _row_stride(t[:1, :1, :8], "t") == 8
    assert _row_stride(torch.zeros(1, 16).expand(5, 16), "t") == 0    # refused by the call
    for bad in (t[:, :3], t.transpose(1, 2)):
        with pytest.raises(ValueError):
            _row_stride(bad, "t")


@pytest.mark.parametrize("gone", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_package_needs_no_private_part_of_torch(gone):
    """Imported on a torch without its private stream and device calls, it
    takes the public ones."""
    code = ("import torch\n"
            f"del torch._C.{gone}\n"
            "import prompt_conditioned_keypoint_amd as gkd\n"
            "from prompt_conditioned_keypoint_amd import binding\n"
            "class S: cuda_stream = 77\n"
            "torch.cuda.current_stream = lambda dev=None: S\n"
            f"gone = {gone!r}\n"
            "assert gone != '_cuda_getCurrentRawStream' or binding._raw_stream(0) == 77\n"
            "assert gone != '_cuda_getDevice' or binding._current_device is torch.cuda.current_device\n"
            "print('fine')\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert res.stdout.strip() == "fine", res.stderr
