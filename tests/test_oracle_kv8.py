"""Pins of the 8-bit cache's and the page calls' oracle (CPU)."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as K8


def test_e4m3_table_and_rounding_are_those_of_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(K8.E4M3, codes.view(torch.float8_e4m3fn).float().numpy())
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 100, rng.normal(size=2000) * 2.0 ** -8, (K8.E4M3[:126] + K8.E4M3[1:127]) / 2,
                        K8.E4M3[:127], -K8.E4M3[:127], [0.0, 448.0, 2.0 ** -10, 2.0 ** -9, 1.5 * 2.0 ** -9]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.as_tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(K8.encode(x), want)


@pytest.mark.parametrize("amax,s", [(0.0, 1.0), (448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (224.5, 1.0), (1.75, 2.0 ** -8),
                                    (1.0, 2.0 ** -8), (1e-44, 2.0 ** -126), (3.38e38, 2.0 ** 120)])
def test_page_scale(amax, s):
    assert K8.page_scale(amax) == s


def test_append_requantises_kept_rows_and_leaves_the_rest():
    codes, scale = np.zeros((2, 1, 16, 64), np.uint8), np.ones((2, 1), np.float32)
    K8.append_request(codes, scale, [1, 0], 0, np.full((3, 1, 64), 1.0))
    assert scale[1, 0] == 2.0 ** -8 and (K8.E4M3[codes[1, 0, :3]] == 256).all()
    codes[1, 0, 5:] = 0x7F
    K8.append_request(codes, scale, [1, 0], 3, np.full((1, 1, 64), 3.0))       # 3 / 448 -> 2^-7
    assert scale[1, 0] == 2.0 ** -7 and (K8.E4M3[codes[1, 0, :3]] == 128).all() and (K8.E4M3[codes[1, 0, 3]] == 384).all()
    assert (codes[1, 0, 5:] == 0x7F).all() and (codes[0] == 0).all() and scale[0, 0] == 1
    K8.append_request(codes, scale, [1, 0], 2, np.full((1, 1, 64), 0.5))       # the large row is gone again
    assert scale[1, 0] == 2.0 ** -8 and (K8.E4M3[codes[1, 0, :2]] == 256).all()


def test_alloc_and_release_are_inverse_and_serve_in_order():
    table = np.full((3, 4), -1, np.int32)
    free, held = np.array([10, 11, 12, 13, 14, -1, -1], np.int32), np.zeros(3, np.int32)
    t, h, c, g, slots = K8.alloc_pages(table, [0, 0, 0], [17, 33, 1], 40, held, free, 5)
    assert g.tolist() == [1, 1, 0] and h.tolist() == [2, 3, 0] and c == 0
    assert t[0, :2].tolist() == [14, 13] and t[1, :3].tolist() == [12, 11, 10]
    assert slots[0, :17].tolist() == [14 * 16 + i for i in range(16)] + [13 * 16] and (slots[0, 17:] == -1).all() and (slots[2] == -1).all()
    f, h2, c2 = K8.release_pages(t, [0, 16, 0], h, free, c)
    assert c2 == 4 and f[:4].tolist() == [14, 13, 11, 10] and h2.tolist() == [0, 1, 0]
