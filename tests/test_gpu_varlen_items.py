"""Packed prefill of batches whose rows select more blocks than they are long: short sequences and cached prefixes, where the
work list holds an item for every selected block."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_varlen import _cfg, _check  # noqa: E402

BATCHES = [
    # name, query lengths, cached prefixes, H_q, H_kv, d_h, d_idx, k
    ("three_chunks", (200, 77, 640), (1024, 0, 384), 8, 2, 128, 32, 4),
    ("one_token_each", (1,) * 600, (0,) * 600, 4, 2, 64, 32, 1),
    ("steps_on_prefixes", (1, 3, 2) * 10, (2048, 1024, 4096) * 10, 16, 4, 128, 64, 16),
    ("windows", (700, 1, 0, 3000, 5), (12800, 0, 256, 6400, 128), 4, 2, 64, 32, 16),
]


@pytest.mark.parametrize("batch", BATCHES, ids=[b[0] for b in BATCHES])
def test_more_blocks_than_rows(batch):
    name, lens, prefix, H_q, H_kv, d_h, d_idx, k = batch
    cfg = _cfg(name, lens, H_q, H_kv, d_h, d_idx, k, prefix)
    _check(cfg, np.arange(cfg.T) if cfg.T <= 1000 else np.unique(np.linspace(0, cfg.T - 1, 500).astype(int)))
