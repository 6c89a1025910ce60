"""Pins of the paged-cache oracle: torch's own e4m3 conversion, steps of the allocator
worked by hand, and closed forms of the attention."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged_cache as pc


def test_e4m3_values_and_rounding_against_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    np.testing.assert_array_equal(pc.e4m3_values(),
                                  codes.view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.integers(-14, 9, 20000)),
                        pc.e4m3_values()[:127], -pc.e4m3_values()[:127],
                        (pc.e4m3_values()[:126] + pc.e4m3_values()[1:127]) / 2,  # ties
                        [0.0, -0.0, 2.0 ** -10, 2.0 ** -11, 448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(pc.e4m3_encode(x), want)
    np.testing.assert_array_equal(pc.e4m3_encode([np.inf, -np.inf, np.nan, 1e9]),
                                  [0x7E, 0xFE, 0x7F, 0x7E])


def test_page_scale():
    assert pc.page_scale(448.0) == 1.0 and pc.page_scale(448.0001) == 2.0
    assert pc.page_scale(224.0) == 0.5 and pc.page_scale(0.0) == 2.0 ** -120
    assert pc.page_scale(1e-40) == 2.0 ** -120


def test_page_tables_by_hand():
    # pages of 4; request 0 grows 3 -> 5 (one page), 1 gives back 9 -> 4 (two pages), 2
    # starts with 6 tokens (two pages), 3 idles, 4 wants one page more than is left
    table = np.full((5, 3), -1)
    table[0, 0], table[1], table[3, 0] = 7, [1, 2, 3], 5
    ring = np.array([10, 11, -1, -1, -1, -1, 8, 9])       # head 6: 8, 9, 10, 11
    out = pc.page_tables([3, 9, 0, 2, 0], [2, -5, 6, 0, 5], table, ring, [6, 4], 14, 4)
    assert out["seq_len"].tolist() == [5, 4, 6, 2, 0]
    assert out["kv_indptr"].tolist() == [0, 2, 3, 5, 6, 6]
    assert out["kv_indices"].tolist() == [7, 8, 1, 9, 10, 5]
    assert out["tok_indptr"].tolist() == [0, 2, 2, 8, 8, 13]
    # ring of 8 pages: page numbers past it (8..11) hold no slot
    assert out["slots"].tolist() == [31] + [-1] * 13
    assert out["tok_req"].tolist() == [0, 0] + [2] * 6 + [4] * 5 + [-1]
    assert out["cursor"].tolist() == [1, 3, 1]
    assert out["ring"].tolist() == [10, 11, 2, 3, -1, -1, 8, 9]
    assert out["table"][0].tolist() == [7, 8, -1] and out["table"][2].tolist() == [9, 10, -1]


def test_cache_write_growth_is_exact_for_powers_of_two():
    codes = np.zeros((1, 1, 16, 2), np.uint8)
    scale = np.ones((1, 1))
    codes, scale = pc.cache_write(np.array([[[1.0, -2.5]]]), [0], codes, scale, 16, False)
    assert scale[0, 0] == 2.0 ** -7                        # 2.5 <= 448 / 128
    codes, scale = pc.cache_write(np.array([[[1000.0, 0.0]]]), [1], codes, scale, 16, False)
    assert scale[0, 0] == 4.0
    v = pc.e4m3_values()[codes[0, 0]] * 4.0
    assert v[0].tolist() == [1.0, -2.5] and v[1, 0] == 1024.0  # 250 -> 256


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((32, 128)), rng.standard_normal((32, 128))
    there = np.ones(32, bool)
    q = rng.standard_normal(128)
    o, av, _ = pc.attend(0 * q, k, v, there, 32, None, 16, 0.1)
    np.testing.assert_allclose(o, v.mean(0), atol=1e-14)   # equal scores: the mean
    np.testing.assert_allclose(av, np.abs(v).mean(0), atol=1e-14)
    o, _, _ = pc.attend(q, k, v, there, 1, None, 16, 0.1)
    np.testing.assert_allclose(o, v[0])                    # one token: its value
    assert not pc.attend(q, k, v, there, 0, None, 16, 0.1)[0].any()
    assert not pc.attend(q, k, v, ~there, 32, None, 16, 0.1)[0].any()
    a = pc.attend(q, k, v, there, 20, [1, -1, 2], 16, 0.1)[0]   # slot 1's first 4 tokens
    b = pc.attend(q, k[16:20], v[16:20], there[:4], 4, None, 4, 0.1)[0]
    np.testing.assert_allclose(a, b)
    o, _, _ = pc.attend(q, k, v, there, 32, None, 16, 0.1, slope=1e4)
    np.testing.assert_allclose(o, v[31])                   # a steep slope: the last token
    o, _, _ = pc.attend(q, k, v, there, 32, None, 16, 1e9, softcap=1e-9)
    np.testing.assert_allclose(o, v.mean(0), atol=1e-8)    # a tiny cap: the mean
