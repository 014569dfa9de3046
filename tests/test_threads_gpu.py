"""Calls from threads other than the one that began."""
from __future__ import annotations

import threading

import pytest
import torch

gpu = pytest.mark.gpu
BF = torch.bfloat16
CALLS = 3000


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


def randn(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


def block_forward(dsa, T, st):
    """The C call with its arguments made before, so that it is a thread's
    first CUDA call, and threads meet inside the library and not in Python."""
    q, k = randn(1, 1, 4, 64), randn(T, 1, 1, 64)
    ids = torch.zeros((1, 1, 8), dtype=torch.int32, device="cuda")
    o, lse, ws = dsa.dsa_block_attn_fwd(q, k, k, ids, 16, 0.1, local_blocks=1)
    args = (q.data_ptr(), k.data_ptr(), k.data_ptr(), None, 1, 1, 4, 1, 64, T,
            ids.data_ptr(), 1, 8, 16, 1, None, 0.1, o.data_ptr(),
            lse.data_ptr(), ws.data_ptr(), ws.numel(), st.cuda_stream)
    return lambda lib: lib.dsa_block_attn_fwd(*args), (o, q, k, ids, lse, ws)


def block_backward(dsa, T, st):
    q, k = randn(1, 1, 4, 64), randn(T, 1, 1, 64)
    ids = torch.zeros((1, 1, 8), dtype=torch.int32, device="cuda")
    o, lse, _ = dsa.dsa_block_attn_fwd(q, k, k, ids, 16, 0.1, local_blocks=1)
    gq, gk, gv, ws = dsa.dsa_block_attn_bwd(q, k, k, o, lse, o, ids, 16, 0.1,
                                            local_blocks=1)
    args = (q.data_ptr(), k.data_ptr(), k.data_ptr(), None, o.data_ptr(),
            lse.data_ptr(), o.data_ptr(), 1, 1, 4, 1, 64, T, ids.data_ptr(), 1,
            8, 16, 1, None, 0.1, gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
            ws.data_ptr(), ws.numel(), st.cuda_stream)
    return (lambda lib: lib.dsa_block_attn_bwd(*args),
            (gk, q, k, ids, o, lse, gq, gv, ws))


def indexer(dsa, S, H, S_kv, topk, st):
    q, k = randn(S, 1, H, 128), randn(S_kv, 1, 128)
    w = torch.ones((S, 1, H), device="cuda")
    sc, idx, ws = dsa.dsa_indexer_fwd(q, k, w, 1, topk)
    args = (q.data_ptr(), k.data_ptr(), w.data_ptr(), S, 1, H, 128, S_kv, 1,
            topk, None, None, idx.data_ptr(), sc.data_ptr(), ws.data_ptr(),
            ws.numel(), st.cuda_stream)
    return lambda lib: lib.dsa_indexer_fwd(*args), (idx, q, k, w, sc, ws)


def indexer_backward(dsa, st):
    q, k = randn(8, 1, 64, 128), randn(32, 1, 128)
    w, gs = torch.ones((8, 1, 64), device="cuda"), torch.ones((1, 8, 4),
                                                             device="cuda")
    idx = torch.zeros((1, 8, 4), dtype=torch.int32, device="cuda")
    gq, gk, gw, ws = dsa.dsa_indexer_bwd(q, k, w, 1, idx, gs)
    args = (q.data_ptr(), k.data_ptr(), w.data_ptr(), 8, 1, 64, 128, 32, 1, 4,
            None, idx.data_ptr(), gs.data_ptr(), gq.data_ptr(), gk.data_ptr(),
            gw.data_ptr(), ws.data_ptr(), ws.numel(), st.cuda_stream)
    return (lambda lib: lib.dsa_indexer_bwd(*args),
            (gq, q, k, w, gs, idx, gk, gw, ws))


def latent(dsa, st):
    q, c = randn(4, 1, 64, 128), randn(32, 1, 128)
    idx = torch.zeros((1, 4, 8), dtype=torch.int32, device="cuda")
    o, lse, ws = dsa.dsa_sparse_mla_fwd(q, c, idx, 0.1)
    args = (q.data_ptr(), c.data_ptr(), idx.data_ptr(), 4, 1, 64, 128, 32, 8,
            0.1, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
            st.cuda_stream)
    return lambda lib: lib.dsa_sparse_mla_fwd(*args), (o, q, c, idx, lse, ws)


FIRST = {
    "block forward": lambda d, st: block_forward(d, 64, st),
    "block backward": lambda d, st: block_backward(d, 64, st),
    "selection": lambda d, st: indexer(d, 1, 64, 64, 8, st),
    "one kernel": lambda d, st: indexer(d, 8, 64, 8192, 8, st),
    "indexer backward": indexer_backward,
    "latent attention": latent,
}


@gpu
@pytest.mark.parametrize("name", FIRST)
def test_a_threads_first_cuda_call(dsa, name):
    """A thread that has made no CUDA call has no context yet."""
    lib = dsa.load_library()
    st = torch.cuda.Stream()
    call, tensors = FIRST[name](dsa, st)
    want = tensors[0].clone()
    tensors[0].zero_()
    torch.cuda.synchronize()
    codes = []
    t = threading.Thread(target=lambda: codes.append(call(lib)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [0]
    assert torch.equal(tensors[0], want)


PAIRS = {
    "block forward": lambda d, a, b: (block_forward(d, 64, a),
                                      block_forward(d, 16 * 16384, b)),
    "block backward": lambda d, a, b: (block_backward(d, 64, a),
                                       block_backward(d, 16 * 8192, b)),
    # the selection's rows, and the one-kernel forward's candidates
    "selection": lambda d, a, b: (indexer(d, 1, 64, 64, 8, a),
                                  indexer(d, 1, 64, 16384, 8, b)),
    "one kernel": lambda d, a, b: (indexer(d, 8, 64, 8192, 8, a),
                                   indexer(d, 8, 64, 8192, 2048, b)),
}


@gpu
@pytest.mark.parametrize("pair", PAIRS)
def test_two_threads_with_contexts_of_different_lengths(dsa, pair):
    """Longer contexts need more shared memory, whose limit is the kernel's:
    one thread's call must not lower it before the other's launch."""
    lib = dsa.load_library()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = PAIRS[pair](dsa, *streams)
    torch.cuda.synchronize()
    codes = [set(), set()]

    def work(i):
        for _ in range(CALLS):
            codes[i].add(calls[i][0](lib))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]
