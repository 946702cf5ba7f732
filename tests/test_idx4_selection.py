"""What the selection loses to 4-bit index keys, as the documents state it (CPU, 64
bits): the share of the chosen blocks that the 16-bit keys also choose, over the
repository's synthetic workloads (queries of normal values, normalised keys).

The stated shares are means over 32 rows; those of single rows lie within 0.025 of
them, so that the mean of 12 other rows is within three times 0.025 / sqrt(12) = 0.022
unless rows deviate more than they were seen to; 0.03 is asked."""
from __future__ import annotations

import numpy as np
import pytest

import synth
from attn_ref import dequantise, quantise


def _f64(bits):
    return synth.bf16_bits_to_f32(bits).astype(np.float64)


def _round4(x):
    return np.concatenate([dequantise(*quantise(x[i:i + 4096])) for i in range(0, len(x), 4096)])


@pytest.mark.parametrize("n,k,share", [(2048, 512, 0.91), (16384, 512, 0.85)])
def test_blocks_chosen_by_both(n, k, share):
    rng = np.random.default_rng(n)
    q, keys = _f64(synth.draw_q(rng, 12)).reshape(12, 4, 128), _f64(synth.draw_normalised_keys(rng, n))
    q4, keys4 = _round4(q.reshape(-1, 128)).reshape(q.shape), _round4(keys)
    s, s4 = (sum(np.maximum(a[:, h] @ b.T, 0.0) for h in range(4)) for a, b in ((q, keys), (q4, keys4)))
    best, best4 = (np.argsort(-x, axis=1, kind="stable")[:, :k] for x in (s, s4))
    both = np.mean([np.isin(a, b).mean() for a, b in zip(best4, best)])
    assert abs(both - share) < 0.03
    kept = np.mean([s[r, best4[r]].sum() / s[r, best[r]].sum() for r in range(len(s))])
    first = np.mean([np.isin(best[r, :k // 4], best4[r]).mean() for r in range(len(s))])
    assert kept > 0.98 and first > 0.995
