"""Refusals of the FP8 projection and read-back calls: status codes of the C ABI before any launch, and the binding's
checks, without a GPU."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
A16, ODD = 0x1000, 0x1008                # addresses that are never read: aligned to 16 bytes, and not


@pytest.fixture(scope="module")
def csa():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import compressed_sparse_attention_18_b200 as m
    return m


def test_mirrors_match_the_c_structs(csa, tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = {"csa_quant_fp8_args": csa.QuantFp8Args, "csa_gemm_fp8_args": csa.GemmFp8Args, "csa_unpack_args": csa.UnpackArgs}
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include "csa.h"\nint main(void){' +
                   "".join(f'printf("%zu\\n", sizeof({n}));' for n in names) + "return 0;}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "sz")], check=True)
    got = subprocess.run([str(tmp_path / "sz")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(t) for t in names.values()]


def quant(csa, **kw):
    a = csa.QuantFp8Args(ctypes.sizeof(csa.QuantFp8Args), 4, 256, 1, A16, A16, A16)
    for k, v in kw.items():
        setattr(a, k, v)
    return csa._lib.csa_quant_fp8(ctypes.byref(a), None)


def test_quant_refusals(csa):
    assert quant(csa, struct_size=8) == INVALID
    assert quant(csa, rows=-1) == INVALID and quant(csa, K=0) == INVALID
    assert quant(csa, block_rows=64) == INVALID and quant(csa, block_rows=0) == INVALID
    assert quant(csa, K=264) == UNSUPPORTED
    assert quant(csa, src=None) == INVALID and quant(csa, codes=None) == INVALID and quant(csa, scales=None) == INVALID
    assert quant(csa, src=ODD) == UNSUPPORTED and quant(csa, codes=ODD) == UNSUPPORTED
    assert quant(csa, rows=0, src=None, codes=None, scales=None) == OK


def gemm(csa, W=(A16, None), W_scales=(A16, None), out=(A16, None), **kw):
    a = csa.GemmFp8Args(ctypes.sizeof(csa.GemmFp8Args), 4, 64, 256, A16, A16)
    for i in range(2):
        for name, v in (("W", W), ("W_scales", W_scales), ("out", out)):
            setattr(a, f"{name}{i}", v[i])
    for k, v in kw.items():
        setattr(a, k, v)
    return csa._lib.csa_gemm_fp8(ctypes.byref(a), None)


def test_gemm_refusals(csa):
    assert gemm(csa, struct_size=8) == INVALID
    assert gemm(csa, M=-1) == INVALID and gemm(csa, N=0) == INVALID and gemm(csa, K=0) == INVALID
    assert gemm(csa, K=264) == UNSUPPORTED and gemm(csa, N=60) == UNSUPPORTED
    for bad in ("x", "x_scales"):
        assert gemm(csa, **{bad: None}) == INVALID
    assert gemm(csa, W=(None, None)) == INVALID and gemm(csa, out=(None, None)) == INVALID
    assert gemm(csa, W_scales=(None, None)) == INVALID
    # a second weight needs its scales and an output of its own; without one there is none of them
    assert gemm(csa, W=(A16, A16)) == INVALID
    assert gemm(csa, W=(A16, A16), W_scales=(A16, A16), out=(A16, A16)) == INVALID
    assert gemm(csa, out=(A16, 2 * A16)) == INVALID and gemm(csa, W_scales=(A16, A16)) == INVALID
    assert gemm(csa, x=ODD) == UNSUPPORTED and gemm(csa, W=(ODD, None)) == UNSUPPORTED
    assert gemm(csa, out=(ODD, None)) == UNSUPPORTED
    assert gemm(csa, M=0, x=None, x_scales=None, W=(None, None), W_scales=(None, None), out=(None, None)) == OK


def unpack(csa, fn, **kw):
    a = csa.UnpackArgs(ctypes.sizeof(csa.UnpackArgs), 2, 3, 512, 64, 8, 1.0, A16, A16, A16, None, None, A16)
    pages = kw.pop("pages", None)
    if pages:
        a.pages = csa.PageMap(*pages)
    for k, v in kw.items():
        setattr(a, k, v)
    return getattr(csa._lib, fn)(ctypes.byref(a), None)


@pytest.mark.parametrize("fn", ["csa_unpack_fp4", "csa_unpack_fp8_window"])
def test_unpack_refusals(csa, fn):
    assert unpack(csa, fn, struct_size=8) == INVALID
    for k in ("B", "n", "n_max"):
        assert unpack(csa, fn, **{k: -1}) == INVALID
    assert unpack(csa, fn, d=0) == INVALID and unpack(csa, fn, d_rope=600) == INVALID
    assert unpack(csa, fn, d=512 + 8) == UNSUPPORTED and unpack(csa, fn, d=512 + 4, d_rope=68) == UNSUPPORTED
    for k in ("codes", "scales", "rope", "out"):
        assert unpack(csa, fn, **{k: None}) == INVALID
    assert unpack(csa, fn, row0=A16, idx=A16) == INVALID
    for k in ("codes", "rope", "out"):
        assert unpack(csa, fn, **{k: ODD}) == UNSUPPORTED
    assert unpack(csa, fn, n=0, codes=None, scales=None, rope=None, out=None) == OK


def test_unpack_formats(csa):
    assert unpack(csa, "csa_unpack_fp4", global_scale=0.0) == INVALID
    assert unpack(csa, "csa_unpack_fp4", global_scale=float("nan")) == INVALID
    assert unpack(csa, "csa_unpack_fp4", pages=(A16, 100, 1, 1)) == UNSUPPORTED        # pages of a multiple of 128
    assert unpack(csa, "csa_unpack_fp4", pages=(A16, 128, 1, 1), n_max=129) == INVALID  # too few pages
    assert unpack(csa, "csa_unpack_fp8_window", pages=(A16, 128, 1, 1)) == UNSUPPORTED  # windows are not paged
    assert unpack(csa, "csa_unpack_fp8_window", d=96 + 64) == UNSUPPORTED               # blocks of 64 channels


def test_binding_refuses_before_the_call(csa):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(csa.CSAError):
        csa.quant_fp8(x)                                         # not on a CUDA device
    with pytest.raises(csa.CSAError):
        csa.quant_fp8(x.float())
    codes, scales = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    with pytest.raises(csa.CSAError):
        csa.Fp8Blocks(codes, scales, 64)
    with pytest.raises(csa.CSAError):
        csa.Fp8Blocks(codes, scales[:, :1], 1)
    with pytest.raises(csa.CSAError):
        csa.Fp8Blocks(codes.float(), scales, 1)
    a, w = csa.Fp8Blocks(codes, scales, 1), csa.Fp8Blocks(codes, scales[:1].contiguous(), 128)
    with pytest.raises(csa.CSAError):
        csa.gemm_fp8(a, a)                                       # a weight has blocks of 128 rows
    with pytest.raises(csa.CSAError):
        csa.gemm_fp8(w, w)
    with pytest.raises(csa.CSAError):
        csa.gemm_fp8(a, csa.Fp8Blocks(codes[:, :128].contiguous(), scales[:1, :1].contiguous(), 128))
    with pytest.raises(csa.CSAError):
        csa.gemm_fp8(a, codes)
    with pytest.raises(csa.CSAError):
        csa.gemm_fp8(a, w, out2=x)
    with pytest.raises(csa.CSAError):
        csa.compress(x=x[None], W_kv=w, W_g=x, b_pos=scales, ratio=4)   # both weights are FP8, or none
    cache = csa.PackedCache(1, 4, 512, 64, "cpu")
    ids = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(csa.CSAError):
        csa.unpack_fp4(cache)
    with pytest.raises(csa.CSAError):
        csa.unpack_fp4(cache, idx=ids, row0=ids[:, 0])
    with pytest.raises(csa.CSAError):
        csa.unpack_fp4(cache, idx=ids, n=3)
    with pytest.raises(csa.CSAError):
        csa.unpack_fp4(cache, idx=ids.long())
    with pytest.raises(csa.CSAError):
        csa.unpack_fp4(cache, row0=ids)
