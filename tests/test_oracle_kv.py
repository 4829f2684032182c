"""The cache and attention oracle against hand-made cases (CPU)."""
import math

import numpy as np
import pytest

from oracle import kv_oracle as KO


def test_plan_by_hand():
    table = np.full((4, 4), -1, np.int32)
    table[0, :1], table[1, :2], table[3, :2] = [7], [8, 9], [5, 6]
    ring = np.array([20, 21, 22, -1, -1, 19], np.int32)  # head 5: 19, 20, 21, 22
    r = KO.plan([16, 20, 0, 32], [1, 12, 3, -1], 16, 16, ring, [5, 4], table)
    assert r["seq_len"].tolist() == [17, 32, 3, 0]
    assert r["q_start"].tolist() == [0, 1, 13, 16, 16]
    assert r["block_table"][0].tolist() == [7, 19, -1, -1] and r["block_table"][2, 0] == 20
    assert r["slot"].tolist() == [19 * 16] + [9 * 16 + 4 + i for i in range(12)] + [20 * 16 + i for i in range(3)]
    assert r["position"].tolist() == [16] + list(range(20, 32)) + [0, 1, 2]
    assert r["free_state"].tolist() == [1, 4, 0]  # two taken, two given back
    assert r["free_pages"].tolist() == [20, 21, 22, 5, 6, 19]


def test_plan_refuses_without_overtaking():
    table = np.full((3, 8), -1, np.int32)
    r = KO.plan([0, 0, 0], [40, 100, 16], 156, 16, np.arange(6, dtype=np.int32), [0, 5], table)
    assert r["seq_len"].tolist() == [40, 0, 0]          # 3 pages, then 7 of 2 left; the last may not overtake
    assert r["free_state"].tolist() == [3, 2, 8]
    assert (r["slot"][40:] == -1).all() and (r["block_table"][1:] == -1).all()


def test_append_by_hand():
    q = np.full((2, 1, 16, 64), 99, np.int8)
    scale = np.full((2, 1), 5.0, np.float32)
    x = np.zeros((2, 1, 64), np.float16)
    x[0, 0, 0], x[0, 0, 1], x[1, 0, 2] = 127, -63.5, 1
    q1, s1 = KO.append(q, scale, x, [16, 17])            # opens page 1: its old scale does not count
    assert s1[1, 0] == 1 and q1[1, 0, 0, :2].tolist() == [127, -64] and q1[1, 0, 1, 2] == 1
    y = np.zeros((1, 1, 64), np.float16)
    y[0, 0, 5] = 254
    q2, s2 = KO.append(q1, s1, y, [18])                  # the scale doubles: earlier tokens are rounded again
    assert s2[1, 0] == 2 and q2[1, 0, 0, :2].tolist() == [64, -32] and q2[1, 0, 1, 2] == 0 and q2[1, 0, 2, 5] == 127
    y[0, 0, 6] = np.inf
    q3, s3 = KO.append(q2, s2, y, [19])
    assert math.isnan(s3[1, 0]) and (q3[1, 0, :4] == 0).all()


@pytest.mark.parametrize("new,seq", [(1, 1), (1, 37), (3, 3), (5, 40), (4, 2)])
def test_attention_against_dense_softmax(new, seq):
    rng = np.random.default_rng(new * 100 + seq)
    k = rng.integers(-127, 128, (4, 2, 16, 64)).astype(np.int8)
    v = rng.integers(-127, 128, (4, 2, 16, 64)).astype(np.int8)
    ks, vs = rng.uniform(0.01, 0.02, (4, 2)).astype(np.float32), rng.uniform(0.01, 0.02, (4, 2)).astype(np.float32)
    q = rng.standard_normal((new, 4, 64)).astype(np.float16)
    table = np.array([[2, 0, 3]])
    out, lse, _ = KO.attention(k, v, ks, vs, q, [0, new], [seq], table, 0.125)
    kd = (k[[2, 0, 3]] * ks[[2, 0, 3]][:, :, None, None]).transpose(1, 0, 2, 3).reshape(2, 48, 64)[:, :seq]
    vd = (v[[2, 0, 3]] * vs[[2, 0, 3]][:, :, None, None]).transpose(1, 0, 2, 3).reshape(2, 48, 64)[:, :seq]
    for i in range(new):
        see = seq - new + i + 1
        for h in range(4):
            if see <= 0:
                assert (out[i, h] == 0).all() and lse[i, h] == -np.inf
                continue
            w = np.exp(0.125 * kd[h // 2, :see] @ q[i, h].astype(np.float64))
            assert np.allclose(out[i, h], (w / w.sum()) @ vd[h // 2, :see], rtol=1e-5, atol=1e-7)
            assert abs(lse[i, h] - math.log(w.sum())) < 1e-5
