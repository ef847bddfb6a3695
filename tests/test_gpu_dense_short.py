"""The dense comparator on ragged batches with fewer 16-key blocks than CTAs:
some CTAs hold no block, and pieces span them."""
import numpy as np
import pytest
import torch

import oracle
import synth
import stochastic_sparse_decode_split_gb300 as santa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lo,hi,B,seed", [(120, 360, 3, 5), (16, 48, 3, 6), (200, 400, 2, 7), (1, 90, 7, 8)])
@pytest.mark.parametrize("fill", [0, 255])
def test_dense_of_fewer_blocks_than_ctas(lo, hi, B, seed, fill):
    """Whatever the workspace held before: the exact result (1e-4 relative L2 per head, as the comparator's other
    tests) and no grid wait that runs out."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    inp = synth.generate(synth.Workload("dense_short", B, 8, 2, 128, hi, "bf16", 1, "systematic", ragged=(lo, hi)), seed)
    t = synth.to_torch(inp)
    p = santa.make_params(t["q"], t["K"], 1, 0, 0, hi, t["kv_offsets"], None, 0.0)
    n = santa.dense_workspace_size(p)
    raw = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
    off = (-raw.data_ptr()) % 256
    ws = raw[off:off + n]
    assert santa.library().santa_workspace_init(santa._ptr(ws), n, santa._stream()) == 0
    ref = oracle.dense(oracle.Problem.from_inputs(inp))
    for _ in range(3):
        out = santa.santa_dense_decode(t["q"], t["K"], t["V"], nk=hi, kv_offsets=t["kv_offsets"], workspace=ws)
        assert santa.get_error(ws) == 0
        rel = np.linalg.norm(out.double().cpu().numpy() - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert rel.max() <= 1e-4
