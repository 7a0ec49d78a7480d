"""8-bit coded operands on the host: sizes and layout of coded buffers, the
refusals of the entry points (all returned before anything is enqueued), and
the oracle's coding rule against hand values."""
import contextlib
import os

import numpy as np
import pytest
import torch

from oracle import coded
from weight_shared_rank_amd import binding

A = 1 << 32  # a fake device address, 256-byte aligned, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIBPATH):
        from weight_shared_rank_amd import build
        build.build(verbose=False)
    return binding.lib()


def align(n, m):
    return -(-n // m) * m


@pytest.mark.parametrize("R,K", [(1, 8), (1, 128), (17, 136), (128, 1152), (129, 5376), (1 << 20, 8)])
def test_code_bytes(L, R, K):
    nb = align(K, 128) // 128
    codes = align(R * nb * 128, 256)
    assert L.weightless_act_code_bytes(R, K) == codes + align(nb * align(R, 16), 256)
    assert L.weightless_weight_code_bytes(R, K) == codes + align(nb * align(align(R, 128) // 128, 4), 256)


@pytest.mark.parametrize("T,K,status,frag", [
    (1, 0, -2, "K"), (1, 12, -2, "multiple of 8"), (1, (1 << 20) + 8, -2, "K"), (-1, 8, -1, "negative"),
    ((1 << 20) + 1, 8, -2, "too large"), (1 << 20, 1 << 18, -2, "2^30 blocks")])
def test_act_shapes_refused(L, T, K, status, frag):
    assert L.weightless_act_code_bytes(T, K) == 0 and frag in binding.last_error()
    assert L.weightless_act_encode(A, T, K, 2 * A, BIG, None) == status and frag in binding.last_error()
    assert L.weightless_act_expand(A, BIG, T, K, 2 * A, None) == status
    assert L.weightless_coded_linear(A, BIG, 64, K, None, 2 * A, BIG, T, 3 * A, 4 * A, BIG, None) == status


@pytest.mark.parametrize("T,nb", [((1 << 20) - 1, 1024), ((1 << 20) - 15, 1024), ((1 << 18) - 3, 4096)])
def test_the_bound_on_blocks_counts_padded_tokens(L, T, nb):
    """T rounded up to 16, times nb, stays below 2^30: refused at it, though T
    itself times nb is below; taken with the next fewer multiple of 16."""
    K = nb * 128
    assert T * nb < 1 << 30 <= align(T, 16) * nb
    assert L.weightless_act_code_bytes(T, K) == 0 and "rounded up to 16" in binding.last_error()
    assert L.weightless_act_encode(A, T, K, 2 * A, 1 << 60, None) == -2
    T = T // 16 * 16
    assert L.weightless_act_code_bytes(T, K) == T * K + nb * T


def test_weight_shapes_refused(L):
    for n, k in ((0, 8), (-1, 8), ((1 << 20) + 1, 8), (8, 4)):
        assert L.weightless_weight_code_bytes(n, k) == 0
        assert L.weightless_weight_encode(A, n, k, 2 * A, BIG, None) == -2
        assert L.weightless_coded_linear(A, BIG, n, k, None, 2 * A, BIG, 1, 3 * A, 4 * A, BIG, None) == -2


def test_no_tokens_is_a_no_op(L):
    assert L.weightless_act_code_bytes(0, 64) >= 256
    assert L.weightless_act_encode(None, 0, 64, None, 0, None) == 0
    assert L.weightless_act_expand(None, 0, 0, 64, None, None) == 0
    assert L.weightless_coded_linear(None, 0, 64, 64, None, None, 0, 0, None, None, 0, None) == 0


def test_encode_arguments_refused(L):
    need = L.weightless_act_code_bytes(4, 256)
    assert L.weightless_act_encode(None, 4, 256, A, need, None) == -1
    assert L.weightless_act_encode(A + 2, 4, 256, 2 * A, need, None) == -1 and "aligned" in binding.last_error()
    assert L.weightless_act_encode(A, 4, 256, 2 * A + 16, need, None) == -1
    assert L.weightless_act_encode(A, 4, 256, 2 * A, need - 1, None) == -5
    assert L.weightless_act_encode(A, 4, 256, A + 1024, need, None) == -1 and "overlap" in binding.last_error()
    assert L.weightless_act_expand(A, need - 1, 4, 256, 2 * A, None) == -5
    assert L.weightless_act_expand(A, need, 4, 256, A + 16, None) == -1 and "overlap" in binding.last_error()
    need = L.weightless_weight_code_bytes(4, 256)
    assert L.weightless_weight_encode(A, 4, 256, 2 * A, need - 1, None) == -5
    assert L.weightless_weight_encode(A + 8, 4, 256, 2 * A, need, None) == -1


def test_coded_linear_arguments_refused(L):
    N, K, T = 512, 256, 64
    wb, xb = L.weightless_weight_code_bytes(N, K), L.weightless_act_code_bytes(T, K)
    nws = L.weightless_coded_linear_workspace_bytes(N, K, T)
    good = dict(w=A, wb=wb, x=2 * A, xc=3 * A, xcb=xb, y=4 * A, ws=5 * A, wsb=nws)

    def call(**kw):
        a = dict(good, **kw)
        return L.weightless_coded_linear(a["w"], a["wb"], N, K, a["x"], a["xc"], a["xcb"], T, a["y"], a["ws"], a["wsb"],
                                         None)
    for bad, status, frag in ((dict(w=None), -1, "weight code"), (dict(w=A + 128), -1, "256-byte"),
                              (dict(wb=wb - 1), -5, "weight code"), (dict(xc=None), -1, "activation code"),
                              (dict(xcb=xb - 1), -5, "activation code"), (dict(x=2 * A + 8), -1, "x must be 16-byte"),
                              (dict(y=None), -1, "y is NULL"), (dict(y=4 * A + 1), -1, "y must be"),
                              (dict(y=3 * A), -1, "overlap"), (dict(y=2 * A), -1, "overlap"),
                              (dict(y=A + 512), -1, "overlap"), (dict(x=3 * A + 16), -1, "overlap"),
                              (dict(xc=A), -1, "overlap")):
        assert call(**bad) == status and frag in binding.last_error(), (bad, binding.last_error())
    if nws:
        for bad, status in ((dict(ws=None), -1), (dict(ws=5 * A + 16), -1), (dict(wsb=nws - 1), -5),
                            (dict(ws=4 * A), -1)):
            assert call(**bad) == status, bad


def test_workspace_is_zero_for_few_tokens_and_small_otherwise(L):
    for n, k in ((21504, 5376), (5376, 21504), (8, 1 << 20), (1 << 20, 8)):
        assert all(L.weightless_coded_linear_workspace_bytes(n, k, T) == 0 for T in (0, 1, 4))
    for T in (5, 16, 17, 64, 333, 2048):
        n = L.weightless_coded_linear_workspace_bytes(5376, 21504, T)
        assert n % 256 == 0 and n <= 16 * T * 5376 * 4


@pytest.mark.parametrize("T", [1, 4, 5, 40])
def test_binding_gives_the_workspace_the_library_asks_for(L, monkeypatch, T):
    """Whatever the library's rule: here every token count needs 512 bytes more
    than it says."""
    class Library:
        def __getattr__(self, name):
            return getattr(L, name)

        def weightless_coded_linear_workspace_bytes(self, N, K, T):
            return L.weightless_coded_linear_workspace_bytes(N, K, T) + 512

        def weightless_coded_linear(self, *args):
            given.append(args[9:11])
            return 0
    given = []
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_scope", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    w, x = binding.WeightCode(5376, 21504, device="cpu"), binding.ActCode(T, 21504, device="cpu")
    for _ in range(2):
        binding.coded_linear(w, x)
    need = L.weightless_coded_linear_workspace_bytes(5376, 21504, T) + 512
    assert len(given) == 2 and all(ptr and size == need for ptr, size in given)


def test_binding_refuses_host_strided_and_mistyped_tensors(L):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (binding.encode_act, binding.encode_weight):
        with pytest.raises(binding.WlError, match="device tensor"):
            f(x)
    with pytest.raises(binding.WlError, match="device tensor"):
        binding.ActCode(4, 64, buf=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(binding.WlError, match="multiple of 8"):
        binding.ActCode(4, 63, device="cpu")


def test_oracle_rule_by_hand():
    assert [coded.exponent(v) for v in (0.0, 448.0, 449.0, 1.75, 1.76, 3.5, 2.0 ** -133, 3.3895e38)] == \
        [0, 0, 1, -8, -7, -7, -118, 120]
    x = np.zeros((2, 130))
    x[0, :4] = [448.0, -1.0, 17.0, 2.0 ** -10]      # e = 0: 17 ties to 16, 2^-10 ties to 0
    x[0, 4] = np.inf
    x[1, 129] = -900.0                              # e = 2: -225 -> -224
    v, e = coded.code(x, 1)
    assert e.tolist() == [[0, 0], [0, 2]]
    assert v[0, :4].tolist() == [448.0, -1.0, 16.0, 0.0] and np.isnan(v[0, 4]) and v[1, 129] == -224.0
    v, e = coded.code(x, 128)
    assert e.tolist() == [[0, 2]] and coded.values(v, e, 128)[1, 129] == -896.0
