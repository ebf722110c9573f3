"""Pins of the oracle's 8-bit form: the e4m3 codes against torch's conversions and hand-worked
values, the scales, the norm and the block-scaled product against brute force."""

import numpy as np
import pytest

import oracle
import q4a_workloads as wl

torch = pytest.importorskip("torch")


def test_e4m3_values():
    got = oracle.e4m3_values(np.arange(256))
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref, equal_nan=True)
    assert oracle.e4m3_value(0x7E) == 448.0 and oracle.e4m3_value(0x01) == 2.0 ** -9
    assert oracle.e4m3_value(0x38) == 1.0 and oracle.e4m3_value(0xC0) == -2.0
    assert np.isnan(oracle.e4m3_value(0x7F)) and np.isnan(oracle.e4m3_value(0xFF))


def test_e4m3_rounding():
    rng = np.random.default_rng(5)
    v = np.concatenate([rng.normal(0, 1, 400), rng.normal(0, 100, 400), rng.normal(0, 2.0 ** -8, 400)])
    v = np.clip(v, -448, 448).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal([oracle.e4m3_round(float(a)) for a in v], ref)
    # ties go to the even mantissa: 1.0625 lies between 1 and 1.125, 1.1875 between 1.125 and 1.25
    assert oracle.e4m3_value(oracle.e4m3_round(1.0625)) == 1.0
    assert oracle.e4m3_value(oracle.e4m3_round(1.1875)) == 1.25
    assert oracle.e4m3_round(2.0 ** -10) == 0 and oracle.e4m3_round(1.5 * 2.0 ** -9) == 2
    assert oracle.e4m3_round(1e30) == 0x7E and oracle.e4m3_round(-1e30) == 0xFE
    assert oracle.e4m3_round(float("nan")) == 0x7F


def test_scales_of_rows_and_blocks():
    rng = np.random.default_rng(6)
    v = rng.normal(0, 1, (130, 272))
    v[3, :128] = 0.0
    s = oracle.e4m3_scales(v)
    assert s.shape == (130, 3)
    assert s[3, 0] == 2.0 ** -100 / 448 and s[7, 2] == np.abs(v[7, 256:]).max() / 448
    b = oracle.e4m3_scales(v, 128)
    assert b.shape == (2, 3)
    assert b[0, 1] == np.abs(v[:128, 128:256]).max() / 448 and b[1, 2] == np.abs(v[128:, 256:]).max() / 448


def test_add_rmsnorm():
    rng = np.random.default_rng(7)
    x, r = rng.normal(0, 1, (3, 96)).astype(np.float32), rng.normal(0, 2, (3, 96)).astype(np.float16)
    w = wl.f32_to_bf16_bits(1 + 0.05 * rng.normal(0, 1, 96))
    n, x_new = oracle.add_rmsnorm(x, r, w, eps=1e-5, shift=0.25)
    stored = (x + r.astype(np.float32)).astype(np.float16).astype(np.float64)
    assert np.array_equal(x_new, stored)
    ref = stored / np.sqrt((stored ** 2).mean(1, keepdims=True) + 1e-5) * (wl.bf16_bits_to_f32(w) + 0.25)
    assert np.allclose(n, ref, rtol=1e-14)
    bits = wl.f32_to_bf16_bits(x)
    assert np.array_equal(oracle.add_rmsnorm(bits)[0], wl.bf16_bits_to_f32(bits).astype(np.float64))
    _, x_new = oracle.add_rmsnorm(x, bits, w)
    assert np.array_equal(x_new, wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(x + wl.bf16_bits_to_f32(bits))))


def test_gemm_e4m3():
    rng = np.random.default_rng(8)
    w, x = (rng.integers(0, 0x7F, (n, 272)).astype(np.uint8) | (rng.integers(0, 2, (n, 272)) << 7).astype(np.uint8)
            for n in (130, 5))
    ws, xs = rng.normal(0, 1, (2, 3)).astype(np.float32), rng.normal(0, 1, (5, 3)).astype(np.float32)
    y, mag = oracle.gemm_e4m3(w, ws, x, xs)
    wv = oracle.e4m3_values(w) * np.repeat(np.repeat(ws.astype(np.float64), 128, 0), 128, 1)[:130, :272]
    xv = oracle.e4m3_values(x) * np.repeat(xs.astype(np.float64), 128, 1)[:, :272]
    assert np.allclose(y, xv @ wv.T, rtol=1e-12, atol=1e-9 * mag.max())
    assert np.allclose(mag, np.abs(xv) @ np.abs(wv).T, rtol=1e-12)
