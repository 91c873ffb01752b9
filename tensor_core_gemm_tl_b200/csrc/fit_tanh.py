"""Coefficients of the tanh polynomials in attention_common.cuh: the minimax fits,
in relative error, of tanh(x) / x by polynomials in u = x^2, of degree 4 on
0 <= x <= 0.5 and of degree 6 on 0 <= x <= 1 (Remez exchange in double
precision).  Prints the coefficients and the error of the polynomials evaluated
in float32.

    python csrc/fit_tanh.py
"""
import numpy as np


def f(u):
    s = np.sqrt(np.maximum(u, 1e-30))
    return np.where(u > 1e-12, np.tanh(s) / s, 1.0 - u / 3.0)


def remez(N, L):
    x = L * L * (1 - np.cos(np.pi * (2 * np.arange(N + 1) + 1) / (2 * (N + 1)))) / 2
    grid = np.linspace(0, L * L, 20001)
    for _ in range(20):
        a = np.hstack([x[:, None] ** np.arange(N), ((-1.0) ** np.arange(N + 1) * f(x))[:, None]])
        c = np.linalg.solve(a, f(x))[:N]
        e = np.polyval(c[::-1], grid) / f(grid) - 1
        # the extrema, alternating in sign
        peaks = []
        for i in range(len(grid)):
            if peaks and (e[i] > 0) == (e[peaks[-1]] > 0):
                if abs(e[i]) > abs(e[peaks[-1]]):
                    peaks[-1] = i
            else:
                peaks.append(i)
        if len(peaks) != N + 1:
            break
        x = grid[peaks]
    return c, np.abs(e).max()


if __name__ == "__main__":
    for N, L in ((5, 0.5), (7, 1.0)):
        c, err = remez(N, L)
        print(f"|x| <= {L}: relative error", err)
        print(", ".join(f"{v:.10g}f" for v in c))
        x = np.linspace(-L, L, 200001).astype(np.float32)
        u, p = x * x, np.full_like(x, np.float32(c[-1]))
        for v in c[-2::-1]:
            p = p * u + np.float32(v)
        print("float32 absolute error", np.abs((p * x).astype(np.float64) - np.tanh(x.astype(np.float64))).max())
