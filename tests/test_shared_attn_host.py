"""Refusals of the shared-prefix attention: status codes of the C ABI before any launch, and the binding's checks,
without a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A16, ODD = 0x1000, 0x1008                # addresses that are never read: aligned to 16 bytes, and not


@pytest.fixture(scope="module")
def csa():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import compressed_sparse_attention_18_b200 as m
    return m


def args(csa, n_prefix=300, prefix=A16, size=None, **kw):
    a = csa.SharedAttnArgs(ctypes.sizeof(csa.SharedAttnArgs) if size is None else size, n_prefix, prefix)
    t = csa.AttnArgs(ctypes.sizeof(csa.AttnArgs), 2, 1, 16, 512, 64, 128, 400, 0, 0, 128, 1.0, 0.0, A16, A16, A16, A16, A16,
                     A16, None, None, None, A16, A16)
    for k, v in kw.items():
        setattr(t, k, v)
    a.attn = t
    return a


def call(csa, ws=None, ws_bytes=0, **kw):
    return csa._lib.hca_shared_attn(ctypes.byref(args(csa, **kw)), ws, ws_bytes, None)


def test_mirror_matches_the_c_struct(csa, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include "csa.h"\nint main(void){printf("%zu\\n", sizeof(csa_shared_attn_args));return 0;}\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "sz")], check=True)
    got = subprocess.run([str(tmp_path / "sz")], capture_output=True, text=True, check=True).stdout
    assert int(got) == ctypes.sizeof(csa.SharedAttnArgs)


def test_refusals(csa):
    assert call(csa, size=8) == INVALID and call(csa, struct_size=8) == INVALID
    assert call(csa, n_prefix=-1) == INVALID and call(csa, n_prefix=401) == INVALID
    assert call(csa, B=-1) == INVALID and call(csa, H=0) == INVALID and call(csa, window=0) == INVALID
    assert call(csa, softmax_scale=-1.0) == INVALID and call(csa, softmax_scale=float("nan")) == INVALID
    assert call(csa, prefix=None) == INVALID and call(csa, q=None) == INVALID and call(csa, kv_codes=None) == INVALID
    assert call(csa, d=128, d_rope=32) == UNSUPPORTED and call(csa, H=65) == UNSUPPORTED
    assert call(csa, flags=1) == UNSUPPORTED and call(csa, flags=2) == UNSUPPORTED
    assert call(csa, prefix=ODD) == UNSUPPORTED and call(csa, q=ODD) == UNSUPPORTED and call(csa, kv_codes=ODD) == UNSUPPORTED
    assert call(csa, B=1 << 20, Nq=64, H=64) == UNSUPPORTED           # 2^32 query rows
    assert call(csa, B=1, Nq=1 << 20, H=64, n_prefix=1 << 21, n_max=1 << 21) == UNSUPPORTED
    assert call(csa) in (WORKSPACE, UNSUPPORTED)                       # (no tensor maps without a driver)
    assert call(csa, B=0) == OK


def test_workspace_sizes(csa):
    size = lambda **kw: csa._lib.csa_shared_attn_workspace_size(ctypes.byref(args(csa, **kw)))  # noqa: E731
    assert size() > 2 * 16 * 512 * 2 and size(B=0) == 0 and size(n_prefix=-1) == 0
    # as many partials as CTAs that share a block of rows: with one block of rows every tile has its own
    row = 2 * 16 * (512 * 2 + 8 * 4 + 4)
    assert size(n_prefix=700, n_max=700) >= 3 * row
    assert size(n_prefix=700, n_max=700) < 4 * row
    # the own keys' partials come on top
    assert size(n_prefix=700, n_max=800) >= 4 * row
    # a long prefix is cut into at most 128 parts
    assert size(n_prefix=1 << 20, n_max=1 << 20) <= 129 * row
    # 2^32 tiles of 128 query rows x 256 keys
    assert size(B=1, Nq=1 << 20, H=64, n_prefix=1 << 21, n_max=1 << 21) == 0
    # without a prefix the call is hca_dense_attn
    a = args(csa, n_prefix=0)
    assert size(n_prefix=0) == csa._lib.csa_attn_workspace_size(ctypes.byref(a.attn), 1)


def test_binding_refuses_before_the_call(csa):
    q = torch.zeros((2, 1, 16, 512), dtype=torch.bfloat16)
    pos, n_c = torch.zeros((2, 1), dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    cache, pre = csa.PackedCache(2, 8, 512, 64, "cpu"), torch.zeros((4, 512), dtype=torch.bfloat16)
    win, p0 = torch.zeros((2, 128, 512), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    good = dict(q=q, q_pos=pos, cache=cache, n_c=n_c, prefix_kv=pre, win_kv=win, win_pos0=p0)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q_pos=pos.int()), dict(q_pos=pos[:1]), dict(n_c=n_c.long()),
                dict(prefix_kv=pre[:, :256]), dict(prefix_kv=pre[None]), dict(cache=csa.PackedCache(1, 8, 512, 64, "cpu")),
                dict(win_kv=win[:1]), dict(win_pos0=None), dict(win_pos0=p0.int()),
                dict(win_kv=csa.Fp8Window(1, 128, 512, 64, "cpu")), dict(out=q.float()), dict(lse=torch.zeros((2, 16)))):
        with pytest.raises(csa.CSAError):
            csa.hca_shared_attn(**{**good, **bad})
    with pytest.raises(csa.CSAError, match="CUDA"):
        csa.hca_shared_attn(**good)
