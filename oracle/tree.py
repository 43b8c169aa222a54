"""Trees of drafted tokens in fp64 -- test infrastructure only.

A tree is a list of parents: -1 a child of the committed prefix, 0 .. t - 1 an earlier node, anything
else no node; a node whose parent is absent is absent.  Every node's result is that of its path
(its ancestors from the root on, then itself) after the committed tokens, so the mixer's
oracle is the sequential recurrence run on every path, and attention is softmax over the
prefix rows and the path's nodes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from .gdn_oracle import mixer

TOKEN_KEYS = ("q", "k", "v", "z", "a", "b")


def _f64(x) -> np.ndarray:
    return np.asarray(torch.as_tensor(x).double().cpu().numpy())


def paths(parent) -> list[list[int]]:
    """For each node the nodes from its root to itself, [] for an absent one."""
    out: list[list[int]] = []
    for t, p in enumerate(parent):
        if p == -1:
            out.append([t])
        elif 0 <= p < t and out[p]:
            out.append(out[p] + [t])
        else:
            out.append([])
    return out


def mixer_tree(inp, parent, state, conv_state) -> dict:
    """The mixer on every path: inp as oracle.mixer's with N*T tokens, parent [N][T] lists, state
    [N][H_v][128][128], conv_state [N][3][C].  out [N*T][H_v][128] (zeros for absent nodes), and state / conv
    of each node that is there, by its token index."""
    N, T = len(parent), len(parent[0])
    H_v = inp["v"].shape[1]
    rows, cu, seqs, toks = [], [0], [], []
    for n in range(N):
        for t, path in enumerate(paths(parent[n])):
            if path:
                rows += [n * T + j for j in path]
                cu.append(len(rows))
                seqs.append(n)
                toks.append(n * T + t)
    out = np.zeros((N * T, H_v, 128))
    states, convs = {}, {}
    if rows:
        sub = {k: inp[k][rows] for k in TOKEN_KEYS}
        sub.update({k: inp[k] for k in ("conv_w", "A_log", "norm_w", "scale")})
        ref = mixer(sub, cu, state_in=state[seqs], conv_in=conv_state[seqs])
        for i, tok in enumerate(toks):
            out[tok] = ref["out"][cu[i + 1] - 1]
            states[tok], convs[tok] = ref["state"][i], ref["conv"][i]
    return {"out": out, "state": states, "conv": convs}


def attention_tree(q, k_tree, v_tree, k_cache, v_cache, cache_len, parent, g=None, scale=None) -> dict:
    """q [N*T][H_q][D], k_tree, v_tree [N*T][H_kv][D], caches [N][cap][H_kv][D].  `out` and, for error bounds, `mass`
    (the same with |v| and the gate) and `shift` (the largest sum |q_i k_i| * scale of a row's scores)."""
    q, k_tree, v_tree = _f64(q), _f64(k_tree), _f64(v_tree)
    _, H, D = q.shape
    Hkv = k_tree.shape[1]
    N, T = len(parent), len(parent[0])
    scale = D ** -0.5 if scale is None else scale
    out, mass, shift = np.zeros_like(q), np.zeros_like(q), np.zeros((N * T, H, 1))
    for n in range(N):
        L = int(cache_len[n])
        kc, vc = _f64(k_cache[n, :L]), _f64(v_cache[n, :L])
        ps = paths(parent[n])
        for t, path in enumerate(ps):
            if not path:
                continue
            idx = [n * T + j for j in path]
            for kv in range(Hkv):
                heads = slice(kv * (H // Hkv), (kv + 1) * (H // Hkv))
                K = np.concatenate([kc[:, kv], k_tree[idx, kv]])
                V = np.concatenate([vc[:, kv], v_tree[idx, kv]])
                s = q[n * T + t, heads] @ K.T * scale
                shift[n * T + t, heads, 0] = np.max(np.abs(q[n * T + t, heads]) @ np.abs(K).T, axis=1) * scale
                with np.errstate(invalid="ignore"):
                    e = np.exp(s - s.max(1, keepdims=True))
                    e /= e.sum(1, keepdims=True)
                    out[n * T + t, heads] = e @ V
                    mass[n * T + t, heads] = e @ np.abs(V)
    if g is not None:
        gate = 1.0 / (1.0 + np.exp(-_f64(g)))
        out, mass = out * gate, mass * gate
    return {"out": out, "mass": mass, "shift": shift}


def rope_frequencies(rotary_dim, base, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, and the factor on cosine and sine."""
    r, half = rotary_dim, rotary_dim // 2
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    theta = np.array([base ** (-i / half) for i in range(half)], dtype=np.float64)
    if scaling == "linear":
        return theta / factor, 1.0
    if scaling == "yarn":
        def pair(beta):
            return r * math.log(original_len / (beta * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), r - 1)
        ramp = np.clip((np.arange(half) - low) / max(high - low, 1e-3), 0, 1)
        return theta * (1 - ramp) + theta / factor * ramp, 0.1 * math.log(factor) + 1.0
    return theta, 1.0


def norm_rope(x, w, positions, rotary_dim, interleaved, theta, amplitude, eps=1e-6) -> dict:
    """x [tokens][heads][D], w [D] or None.  y, and `size`: |y1| + |y2| of the pair each element comes from."""
    x = _f64(x)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * _f64(w)
    y, size = x.copy(), np.abs(x)
    half = rotary_dim // 2
    if half == 0:
        return {"y": y, "size": size}
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + 1 if interleaved else i1 + half
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(theta)[None, :]
    c, s = np.cos(ang)[:, None] * amplitude, np.sin(ang)[:, None] * amplitude
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    size[..., i1] = size[..., i2] = (np.abs(x[..., i1]) + np.abs(x[..., i2])) * amplitude
    return {"y": y, "size": size}
