"""Calls on an explicit stream that is not the current one: what they allocate
comes from that stream's memory, and the results are the current stream's."""
import numpy as np
import pytest
import torch

import harness as H
from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W
from test_gpu_scaled_calls import pool_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()


@pytest.mark.parametrize("as_number", [False, True])
def test_what_a_call_on_another_stream_allocates_is_that_streams(as_number, monkeypatch):
    r = np.random.default_rng(0)
    s, h, d, bs, nb = 3, 4, 64, 16, 24
    kc, vc = (torch.from_numpy(r.standard_normal((nb, h, bs, d))).half().cuda() for _ in range(2))
    q = torch.from_numpy(r.standard_normal((s, h, d))).half().cuda()
    tables = torch.from_numpy(r.permutation(nb).astype(np.int32).reshape(3, 8)).cuda()
    tables[:, 0] = tables[0, 0].clone()
    ctx = torch.tensor([100, 128, 17], dtype=torch.int32, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    group = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    blocks = torch.tensor([1], dtype=torch.int32, device="cuda")
    tokens = torch.from_numpy(r.integers(0, 1000, 300).astype(np.int32)).cuda()
    lens = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    desc = B.cache_desc(kc, vc)
    side = torch.cuda.Stream()
    st = side.cuda_stream if as_number else side

    calls = dict(
        decode=lambda st: B.pkv_paged_attention_decode(desc, q, tables, ctx, 128, 0.125,
                                                       partition_size=32, stream=st),
        static=lambda st: B.pkv_paged_attention_decode_static_ws(desc, q, tables, ctx, 128, 0.125,
                                                                 partition_size=32, stream=st),
        shared=lambda st: B.pkv_paged_attention_decode_shared_prefix(
            desc, q, tables, ctx, 128, group, blocks, 3, 1, 0.125, partition_size=32, stream=st),
        prefill=lambda st: B.pkv_paged_attention_prefill(desc, q, cu, 1, tables, ctx, 128, 0.125,
                                                         stream=st),
        hashes=lambda st: B.pkv_block_hashes(tokens, lens, bs, stream=st))
    torch.cuda.synchronize()
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    for name, call in calls.items():
        out = call(st)
        assert pool_of(out.data_ptr()) == side.cuda_stream, name
        torch.cuda.synchronize()
        assert all(pool_of(t.data_ptr()) == side.cuda_stream for t in made), name
        want = call(None)
        torch.cuda.synchronize()
        assert torch.equal(out, want), name
        made.clear()
