"""Rows whose largest cache value lies within a few fp32 steps of the border between two exponents of a
quantised row, and which exponent an fp32 evaluation of each would choose."""

import numpy as np
import torch

BORDER = 3.5   # 448 * 2^-7: one step more takes the next exponent
EPS = 1e-6


def border_rows(n, first, theta, seed):
    """x [n, 576] fp32, gamma [512] (bf16 values), both in numpy; row i is at position first + i. The
    largest value of even rows is a latent one, of odd rows a rotated one; it is the fp32 input next to
    the border, on one side or the other."""
    rng = np.random.default_rng(seed)
    gamma = torch.from_numpy(1 + 0.1 * rng.standard_normal(512)).to(torch.bfloat16).double().numpy()
    x = np.clip(rng.standard_normal((n, 576)), -1.5, 1.5).astype(np.float32)
    x[:, 512:] = np.clip(x[:, 512:], -1, 1)
    for i in range(n):
        side = rng.random() < 0.5
        if i % 2 == 0:
            j = int(rng.integers(512))
            rest = x[i, :512].astype(np.float64)
            rest[j] = 0.0
            s = (rest ** 2).sum()
            # x^2 g^2 = B^2 ((s + x^2) / 512 + eps)
            value = BORDER * np.sqrt((s / 512 + EPS) / (gamma[j] ** 2 - BORDER ** 2 / 512))
            at = lambda v: v * gamma[j] / np.sqrt((s + v * v) / 512 + EPS)
            place = j
        else:
            angle = (first + i) * theta
            m = int(rng.choice(np.flatnonzero(np.abs(np.cos(angle)) > 0.85)))
            cs, sn = np.cos(angle[m]), np.sin(angle[m])
            other = 0.2 * float(x[i, 512 + 2 * m + 1])
            x[i, 512 + 2 * m + 1] = other
            other = np.float64(x[i, 512 + 2 * m + 1])
            value = (BORDER + other * sn) / abs(cs) if cs > 0 else -(BORDER + other * sn) / abs(cs)
            at = lambda v: v * cs - other * sn
            place = 512 + 2 * m
        v = np.float32(value)
        steps = [v]
        for _ in range(4):
            steps = [np.nextafter(steps[0], np.float32(0))] + steps + [np.nextafter(steps[-1], np.float32(np.sign(v) * 99))]
        sizes = np.abs([at(np.float64(s)) for s in steps])
        under = int(np.flatnonzero(sizes <= BORDER)[-1])
        x[i, place] = steps[under + (1 if side else 0)]
    return x, gamma


def rows_in(kind, x, gamma, first, theta):
    """The cache rows, evaluated in `kind` from angles reduced in fp64."""
    x, g = x.astype(kind), gamma.astype(kind)
    c = x[:, :512] * (kind(1) / np.sqrt((x[:, :512] ** 2).mean(axis=1, keepdims=True) + kind(EPS))) * g
    a = np.remainder((first + np.arange(len(x)))[:, None] * theta[None], 2 * np.pi).astype(kind)
    even, odd = x[:, 512::2], x[:, 513::2]
    k = np.stack([even * np.cos(a) - odd * np.sin(a), even * np.sin(a) + odd * np.cos(a)], axis=2)
    return np.concatenate([c, k.reshape(len(x), 64)], axis=1)


def exponents(rows):
    most = np.abs(rows).astype(np.float64).max(axis=1)
    assert np.all((most > 1.8) & (most < 6.9))
    return np.where(most <= BORDER, -7, -6)
