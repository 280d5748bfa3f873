"""Fits of the bf16 GeLUs' normal-tail polynomial p(u) ~ log2 Phi(-u) on [0, 6], near-minimax
in the absolute error of p (so in the relative error of 2^p), by Lawson's iteratively
reweighted least squares on Chebyshev points: degree 6 for the layer's FFN (gelu_bf16 in
common.hpp), degree 9 for the products with an epilogue (gelu_product in linear.hpp).
Prints the coefficients c0, c1, ... as float32."""
import numpy as np
from scipy.special import log_ndtr

U, N = 6.0, 4000


def fit(degree):
    """(coefficients c0 .. c_degree, max |p - log2 Phi(-u)|)"""
    t = np.cos(np.pi * (np.arange(N) + 0.5) / N)
    u = (t + 1) * U / 2
    f = log_ndtr(-u) / np.log(2)
    A = np.stack([u ** i for i in range(degree + 1)], 1)
    w = np.full(N, 1.0 / N)
    for _ in range(200):
        c, *_ = np.linalg.lstsq(A * np.sqrt(w)[:, None], f * np.sqrt(w), rcond=None)
        e = np.abs(A @ c - f)
        w = w * e
        w /= w.sum()
    return c, np.abs(A @ c - f).max()


if __name__ == "__main__":
    for degree in (6, 9):
        c, err = fit(degree)
        print(f"degree {degree}: max |p - log2 Phi(-u)| = {err:.3g}")
        for i, v in enumerate(np.float32(c)):
            print(f"  c{i} = {float(v):.9g}")
