"""Plain 64-bit numpy implementation of the microscaled 4-bit format and of
Newton-Schulz orthogonalisation, written from their definitions (shares no
code with the library)."""

import math

import numpy as np

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MID = (MAG[1:] + MAG[:-1]) / 2


def code_pitch(K):
    return 16 * -(-K // 32)


def scale_pitch(K):
    return 16 * -(-K // 512)


def quantize(X):
    """X [M, K] float64 -> (codes [M, code_pitch], scales [M, ceil(K/32)])."""
    M, K = X.shape
    nb = -(-K // 32)
    P = np.zeros((M, nb * 32))
    P[:, :K] = X
    P = P.reshape(M, nb, 32)
    codes = np.zeros((M, nb, 32), np.uint8)
    scales = np.zeros((M, nb), np.uint8)
    for i in range(M):
        for b in range(nb):
            x = P[i, b]
            if not np.all(np.isfinite(x)):
                scales[i, b] = 255
                continue
            top = np.max(np.abs(x))
            e = -127 if top == 0 else max(-127, math.frexp(top)[1] - 1 - 2)
            scales[i, b] = e + 127
            m = np.abs(x) * 2.0 ** -e if e > -1000 else x
            c = np.searchsorted(MID, m, side="left")  # m == midpoint: the lower code
            tie = np.isin(m, MID) & (c % 2 == 1)      # ... unless that one is odd
            c = np.minimum(c + tie, 7)
            codes[i, b] = c + 8 * np.signbit(x)
    flat = codes.reshape(M, nb * 32)
    flat[:, K:] = 0
    return (flat[:, 0::2] | (flat[:, 1::2] << 4)).astype(np.uint8), scales


def values(codes, scales, K):
    """float64 values [M, K] of codes [M, >= code_pitch] and scales."""
    nb = -(-K // 32)
    q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)[:, :nb * 32]
    v = np.where(q & 8, -1.0, 1.0) * MAG[q & 7]
    s = scales[:, :nb].astype(np.float64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return (v * np.repeat(f, 32, axis=1))[:, :K]


def newton_schulz(G, steps, a, b, c, eps):
    X = G / (np.linalg.norm(G) + eps)
    for _ in range(steps):
        if X.shape[0] <= X.shape[1]:
            S = X @ X.T
            X = a * X + (b * S + c * (S @ S)) @ X
        else:
            S = X.T @ X
            X = a * X + X @ (b * S + c * (S @ S))
    return X


def newton_schulz_step_bound(G, a, b, c, eps):
    """Elementwise bound on the error of ONE step whose products take FP16
    operands: u = 2^-11 is half an FP16 step relative to the value, t the
    absolute rounding below FP16's normal range (half of 2^-24, over the
    power-of-two scales 2^12 of S and 2^10 of B; X has at least scale 1), f
    the fp32 sums (K + 4 roundings of 2^-23 at most, K <= 4096), and the bf16
    result's own half step 2^-8."""
    u, f = 2.0 ** -11, 4100 * 2.0 ** -23
    X = G / (np.linalg.norm(G) + eps)
    if X.shape[0] > X.shape[1]:
        return newton_schulz_step_bound(G.T, a, b, c, eps).T
    tx, ts, tb = 2.0 ** -25, 2.0 ** -37, 2.0 ** -35
    aX = np.abs(X)
    dX = u * aX + tx
    S = X @ X.T
    aS = aX @ aX.T
    dS = dX @ aX.T + aX @ dX.T + dX @ dX.T + f * aS
    dS = dS + u * (np.abs(S) + dS) + ts
    B = b * S + c * (S @ S)
    aSS = np.abs(S) @ np.abs(S)
    dB = abs(b) * dS + abs(c) * (dS @ np.abs(S) + np.abs(S) @ dS + dS @ dS + f * aSS)
    dB = dB + u * (np.abs(B) + dB) + tb
    out = a * X + B @ X
    d = dB @ aX + np.abs(B) @ dX + dB @ dX + f * (np.abs(B) @ aX) + abs(a) * (2.0 ** -21 * aX + tx)
    return d + 2.0 ** -8 * (np.abs(out) + d) + 1e-30
