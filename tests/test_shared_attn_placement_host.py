"""Where hca_shared_attn attends the sequences' own keys, read off its workspace (which holds a bf16 copy of them when the
prefix kernel takes them), without a GPU: a window buffer longer than the window costs the per-query attention nothing."""
import ctypes

import pytest

A16 = 0x1000                             # an address that is never read


@pytest.fixture(scope="module")
def csa():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import compressed_sparse_attention_18_b200 as m
    return m


def copies_own_keys(csa, B, Nq, H, n_p, own, Wn, window=128):
    """Whether one more window row in the buffer makes the workspace larger by its copies."""
    def size(Wn):
        t = csa.AttnArgs(ctypes.sizeof(csa.AttnArgs), B, Nq, H, 512, 64, 128, n_p + own, 0, Wn, window, 1.0, 0.0, A16, A16, A16,
                         A16, A16, A16, None, A16, A16, A16, A16)
        a = csa.SharedAttnArgs(ctypes.sizeof(csa.SharedAttnArgs), n_p, A16, t)
        return csa._lib.csa_shared_attn_workspace_size(ctypes.byref(a))
    assert Wn >= window and size(Wn) > 0
    return size(Wn + 1) > size(Wn)


@pytest.mark.parametrize("B,Nq,H,n_p,own,Wn", [(1, 4096, 64, 8192, 64, 4223), (2, 2048, 64, 8192, 64, 2175),
                                               (64, 1, 64, 8192, 64, 1024), (128, 1, 16, 512, 500, 640)])
def test_long_window_buffers_stay_with_the_per_query_attention(csa, B, Nq, H, n_p, own, Wn):
    """These took 1.2 to 1.7 times as long in the prefix kernel, which walks the whole buffer."""
    assert not copies_own_keys(csa, B, Nq, H, n_p, own, Wn)


@pytest.mark.parametrize("B,Nq,H,n_p,own,Wn,copied", [
    (2, 1, 16, 260, 3, 128, True), (8, 5, 24, 4099, 70, 132, True), (64, 1, 64, 8192, 64, 128, True),
    (40, 1, 16, 200, 3000, 128, True), (4, 512, 16, 2000, 100, 639, True), (1, 2048, 1, 2000, 64, 2175, True),
    (200, 1, 4, 300, 500, 128, False), (130, 1, 1, 300, 500, 128, False)])
def test_windows_of_their_own_length(csa, B, Nq, H, n_p, own, Wn, copied):
    assert copies_own_keys(csa, B, Nq, H, n_p, own, Wn) == copied
