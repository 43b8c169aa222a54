"""Tree calls at the edges of what they take: rows whose result has to be NaN, trees of very few rows, calls that two threads make at once."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_81_b200 import gdn
from gpu_helpers import OUT_TOL, out_error
from test_gpu_tree import KEYS, attn_case, attn_check, attn_run, delta_case, delta_ref, dev_tree, make_tree

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ gdn_attention_tree

# one sequence cut between many workers, a few sequences, a batch whose units are cut here and whole there
SPLITS = [(1, 3, 24, 4, 256, [3000]), (2, 5, 8, 2, 128, [700, 2100]), (300, 2, 2, 1, 128, [(i * 37) % 300 for i in range(300)])]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N,T,H,Hkv,D,lens", SPLITS)
def test_attention_tree_query_that_is_not_finite_gives_nan(N, T, H, Hkv, D, lens, value):
    """A node's query head with an element that is not finite has scores that no softmax can weigh: NaN by the definition,
    however the work is split, and no other row changes."""
    c = attn_case(N, T, H, Hkv, D, lens, "chain", seed=51)
    clean = attn_run(c).view(N, T, H, D)
    c["q"].view(N, T, H, D)[:, T - 1, H - 1, 7] = value
    out = attn_run(c).view(N, T, H, D)
    assert bool(torch.isnan(out[:, T - 1, H - 1]).all())
    rest = torch.ones(N, T, H, dtype=torch.bool, device="cuda")
    rest[:, T - 1, H - 1] = False
    assert torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("N,T,H,Hkv,D,lens", SPLITS)
def test_attention_tree_row_whose_scores_are_all_minus_infinity_gives_nan(N, T, H, Hkv, D, lens):
    """Every visible score -inf: 0 / 0 by the definition; an absent node's row stays zeros beside it."""
    c = attn_case(N, T, H, Hkv, D, lens, "chain", seed=52)
    c["parent"][:, T - 1] = -2
    c["q"].view(N, T, H, D)[:, 0, 0, 3] = -float("inf")
    c["kc"][..., 3] = c["kc"][..., 3].abs() + 0.125
    c["kt"][..., 3] = c["kt"][..., 3].abs() + 0.125
    out = attn_run(c).view(N, T, H, D)
    assert bool(torch.isnan(out[:, 0, 0]).all()) and bool((out[:, T - 1] == 0).all())
    assert bool(torch.isfinite(out[:, :T - 1, 1:]).all())


@pytest.mark.parametrize("H,Hkv,D", [(1, 1, 128), (24, 4, 256)])
def test_attention_tree_nan_keys_at_the_cache_s_beginning_give_nan(H, Hkv, D):
    """Keys that are NaN in a long cache's first 16 tiles of 128: every node sees them, whichever workers'
    partials they fall into."""
    c = attn_case(1, 2, H, Hkv, D, [6000], "chain", seed=53)
    c["kc"][0, :16 * 128] = float("nan")
    assert bool(torch.isnan(attn_run(c)).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens", [[150], [40] * 200])
def test_attention_tree_key_that_is_not_finite_reaches_its_descendants(value, lens):
    """A node whose key and value are NaN or infinite: NaN for every row that sees it (infinite scores of both signs, or an
    infinite value under a weight of NaN), nothing for the others."""
    N, T, bad, H, D = len(lens), 24, 3, 24, 256
    c = attn_case(N, T, H, 4, D, lens, "holes", seed=9)
    clean = attn_run(c).view(N, T, H, D)
    for x in (c["kt"], c["vt"]):
        x[bad] = value
    out = attn_run(c).view(N, T, H, D)
    hit = torch.zeros(N, T, dtype=torch.bool, device="cuda")
    hit[0] = torch.tensor([bad in p for p in oracle.tree.paths(c["rows"][0])], device="cuda")
    assert bool(hit.any()) and torch.equal(out[~hit], clean[~hit])
    ref = oracle.tree.attention_tree(c["q"][:T].cpu(), c["kt"][:T].cpu(), c["vt"][:T].cpu(), c["kc"][:1].cpu(), c["vc"][:1].cpu(),
                                     lens[:1], c["rows"][:1], c["g"][:T].cpu())["out"]
    want = torch.from_numpy(np.isnan(ref)).cuda()
    assert torch.equal(torch.isnan(out[0])[hit[0]], want[hit[0]])


@pytest.mark.parametrize("lens", [[500], [300] * 150])
def test_attention_tree_whole_tiles_of_lowest_values_and_masked_infinite_scores(lens):
    """Two whole tiles of keys whose scores are about -2e36 before any others, and nodes off the path with infinite scores of both
    signs: each row's weights are those of the keys that it sees.  (A score is a power of two times whole numbers below 2^8
    here, so sums are exact, whatever their order.)"""
    N, T, H, D = len(lens), 6, 4, 128
    c = attn_case(N, T, H, 4, D, lens, "flat", seed=4, gate=False)
    low = -2.0 ** 117  # 128 of them: -2^124 / 128 ** 0.5 = about -1.9e36 each score
    c["q"].fill_(1.0)
    c["kc"][:, :256] = low
    c["kc"][:, 256:] = 0.0
    c["kt"].zero_()
    c["kt"].view(N, T, 4, D)[:, 1] = float("inf")
    c["kt"].view(N, T, 4, D)[:, 4] = -float("inf")
    out = attn_run(c).view(N, T, H, D)
    assert bool(torch.isnan(out[:, 1]).all()) and bool(torch.isfinite(out[:, [0, 2, 3, 5]]).all())
    for n in range(min(N, 3)):
        old = c["vc"][n, 256:lens[n]].double()
        for t in (0, 2, 3, 4, 5):  # uniform weights over the zero scores; node 4's own score weighs nothing
            seen = old if t == 4 else torch.cat([old, c["vt"].view(N, T, 4, D)[n, t].double()[None]])
            want = seen.mean(0)
            # the weights are exactly 1 in bf16, so what is left is the sums' (len 2^-24 of sum |v| each) and the output's rounding
            tol = 2.0 ** -8 * want.abs() + 2 * len(seen) * 2.0 ** -24 * seen.abs().mean(0)
            assert bool(((out[n, t].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("N,T,H,Hkv,D,lens", [(1, 64, 16, 1, 256, [700]), (3, 50, 48, 3, 128, [129, 0, 640]), (2, 3, 64, 64, 128, [257, 30])])
def test_attention_tree_most_heads_of_each_kind(N, T, H, Hkv, D, lens):
    """16 query heads to a KV head at both head sizes, and as many KV heads as query heads."""
    c = attn_case(N, T, H, Hkv, D, lens, "holes", seed=N * T)
    out = attn_run(c)
    attn_check(c, out)
    assert torch.equal(attn_run(c), out)


# ------------------------------------------------------------------ gdn_qk_norm_rope

def test_rope_amplitude_of_the_caller():
    """A factor on cosine and sine that the caller stores in the table."""
    q = torch.randn(9, 3, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 977
    rope = gdn.make_rope(128, 64, scaling="yarn", factor=1.0, original_len=4096)
    want = gdn.qk_norm_rope(rope, q, positions=pos)[0]
    rope.amplitude = 2.0
    got = gdn.qk_norm_rope(rope, q, positions=pos)[0]
    assert torch.equal(got[..., :64], 2 * want[..., :64]) and torch.equal(got[..., 64:], want[..., 64:])


# ------------------------------------------------------------------ gdn_decode_tree

@pytest.mark.parametrize("T,H_v", [(1, 2), (1, 3), (1, 7), (2, 3), (3, 2), (4, 2), (1, 8)])
def test_decode_tree_fewer_rows_than_warps(T, H_v):
    """Many sequences of trees so small that a CTA's warps outnumber its (node, value head) pairs: every repetition the same
    bits, and the results of one sequence alone, whose value heads have a CTA each."""
    N = 400
    c = delta_case(N, T, 1, H_v, "chain", seed=81 + T)
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"])
    for _ in range(40):
        assert torch.equal(gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"]), out)
    n = 40
    sub = dict(c, rows=c["rows"][:n], slot=c["slot"][:n], inp={k: v[:n * T] if k in KEYS else v for k, v in c["inp"].items()})
    assert out_error(out[:n * T], delta_ref(sub)["out"]) <= OUT_TOL
    alone = gdn.decode_tree(c["s"], 1, T, c["parent"][:1].contiguous(), c["d_state"], c["d_conv"], state_slot=c["d_slot"][:1].contiguous())
    assert torch.equal(alone, out[:T])


@pytest.mark.parametrize("value", [float("inf"), 3e38, 1e20, 1e9, 300.0, 120.0])
@pytest.mark.parametrize("N,T,H_k,H_v", [(1, 7, 2, 6), (90, 7, 2, 6), (1, 16, 2, 6), (2, 32, 2, 4), (1, 40, 2, 6), (90, 61, 1, 3)])
def test_decode_tree_gate_that_forgets_everything(N, T, H_k, H_v, value):
    """A decay logit so large that the node's decay is zero: its descendants go on from an empty state, as decoding the
    path token by token does."""
    c = delta_case(N, T, H_k, H_v, "chain", seed=61 + T, a_mean=-2.0)
    at = T // 3
    tok = torch.arange(N) * T + at
    for x in (c["inp"]["a"], c["dev"]["a"]):
        x[tok.to(x.device)] = value
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"])
    assert bool(torch.isfinite(out).all())
    n = min(N, 2)
    sub = dict(c, rows=c["rows"][:n], slot=c["slot"][:n], inp={k: v[:n * T] if k in KEYS else v for k, v in c["inp"].items()})
    sl = sub["slot"].long()
    ref = oracle.tree.mixer_tree(sub["inp"], sub["rows"], c["state"][sl], c["conv"][sl])["out"]
    assert np.isfinite(ref).all()
    assert out_error(out[:n * T], ref) <= OUT_TOL


@pytest.mark.parametrize("T", [1, 5, 8])
@pytest.mark.parametrize("N", [1, 70])
def test_decode_tree_as_many_value_heads_as_key_heads(N, T):
    c = delta_case(N, T, 3, 3, "holes", seed=N + T)
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"])
    t = c["there"].numpy()
    assert bool((out[~c["there"].cuda()] == 0).all())
    assert out_error(out[c["there"].cuda()], delta_ref(c)["out"][t]) <= OUT_TOL


@pytest.mark.parametrize("N,T", [(3, 5), (160, 5), (3, 16), (3, 30), (3, 60), (160, 60)])
def test_a_sequence_without_nodes(N, T):
    """A padded batch: one sequence has no node at all.  Zero rows for it, through both mixers, the others as they were; its
    commits accept nothing, and a node accepted all the same is reported."""
    c = delta_case(N, T, 1, 3, "chain", seed=T)
    want = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"]).view(N, T, -1)
    c["parent"][1] = -2
    for k in KEYS:
        c["dev"][k][T:2 * T] = float("nan")
    out = gdn.decode_tree(c["s"], N, T, c["parent"], c["d_state"], c["d_conv"], state_slot=c["d_slot"]).view(N, T, -1)
    others = torch.arange(N, device="cuda") != 1
    assert bool((out[1] == 0).all()) and torch.equal(out[others], want[others])
    a = attn_case(N, T, 8, 2, 128, [(n * 31) % 200 for n in range(N)], "chain", seed=T)
    want = attn_run(a).view(N, T, -1)
    a["parent"][1] = -2
    a["q"].view(N, T, 8, 128)[1] = float("nan")
    out = attn_run(a).view(N, T, -1)
    assert bool((out[1] == 0).all()) and torch.equal(out[others], want[others])
    for last, bits in ((-1, 0), (0, 128)):
        acc = torch.full((N,), last, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        S, C = c["d_state"].clone(), c["d_conv"].clone()
        gdn.decode_tree_commit(c["s"], N, T, c["parent"], acc, S, C, state_slot=c["d_slot"], err=err)
        slot = int(c["slot"][1])
        assert torch.equal(S[slot], c["d_state"][slot]) and torch.equal(C[slot], c["d_conv"][slot]) and bool(torch.isfinite(S).all())
        assert int(err.item()) == bits
        err.zero_()
        kc, vc = torch.zeros(N, 210, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 210, 2, 128, dtype=torch.bfloat16, device="cuda")
        new = gdn.attn_tree_commit(a["kt"], a["vt"], T, a["parent"], acc, kc, vc, a["len"], cache_len_out=torch.empty_like(a["len"]), err=err)
        assert torch.equal(new, a["len"] + (last + 1) * others.int()) and not bool(kc[1].any()) and int(err.item()) == bits


# ------------------------------------------------------------------ gdn_decode_tree_commit

def test_decode_tree_commit_reads_the_path_s_query_rows():
    """The q channels of the conv state are the path's last three raw q rows: what q holds at the commit counts."""
    T, H_k, H_v = 6, 2, 6
    c = delta_case(1, T, H_k, H_v, "chain", seed=71)
    acc = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    C = c["d_conv"].clone()
    gdn.decode_tree_commit(c["s"], 1, T, c["parent"], acc, c["d_state"].clone(), C, state_slot=c["d_slot"])
    q = c["dev"]["q"].reshape(T, H_k * 128)
    assert torch.equal(C[int(c["slot"][0]), :, :H_k * 128], q[T - 3:])


# ------------------------------------------------------------------ two host threads

CALLERS = r"""
#include <atomic>
#include <functional>
#include <thread>
// a call whose arguments are all integers or addresses: each has its 64-bit slot (x86-64)
struct Call { long long a[13]; };
typedef int (*Fn)(long long, long long, long long, long long, long long, long long, long long, long long, long long, long long,
                  long long, long long, long long);
// two threads, each with its own call, `times` times; the first status that is not 0
extern "C" int two_callers(Fn fn, const Call* calls, int times) {
  std::atomic<int> bad{0}, ready{0};
  auto run = [&](const Call& c) {
    const long long* a = c.a;
    ++ready;
    while (ready < 2) {}
    for (int i = 0; i < times && bad == 0; ++i) {
      const int s = fn(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12]);
      if (s != 0) bad = s;
    }
  };
  std::thread x(run, std::cref(calls[0])), y(run, std::cref(calls[1]));
  x.join();
  y.join();
  return bad;
}
"""


class Call(ctypes.Structure):
    _fields_ = [("a", ctypes.c_longlong * 13)]

    def __init__(self, *args):
        super().__init__((ctypes.c_longlong * 13)(*args))


@pytest.fixture(scope="module")
def two_callers(tmp_path_factory):
    d = tmp_path_factory.mktemp("callers")
    (d / "callers.cpp").write_text(CALLERS)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-o", str(d / "callers.so"), str(d / "callers.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(d / "callers.so"))

    def run(name, a, b, times=20000):
        torch.cuda.synchronize()
        status = lib.two_callers(ctypes.cast(getattr(gdn.load(), name), ctypes.c_void_p), (Call * 2)(a, b), times)
        torch.cuda.synchronize()
        return status
    return run


def no_slots(N, T, H_v):
    """A case whose slots are all out of range, so that the GPU's part of a call is short."""
    c = delta_case(N, T, 1, H_v, "chain", seed=T)
    c["d_slot"] = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    c["acc"] = torch.full((N,), T - 1, dtype=torch.int32, device="cuda")
    c["out"] = torch.ones(N * T, H_v, 128, dtype=torch.bfloat16, device="cuda")
    c["stream"] = torch.cuda.Stream()
    return c


@pytest.mark.parametrize("T", [5, 13, 30, 60])
def test_two_threads_call_decode_tree_with_different_sizes(two_callers, T):
    """Calls of one kernel with different amounts of shared memory (value heads per CTA), from two host threads at once:
    none fails."""
    cases = [no_slots(160, 5, 2), no_slots(160, 5, 8)] if T == 5 else [no_slots(1, T, 8), no_slots(160, T, 8)]
    calls = [Call(ctypes.addressof(c["s"]), c["N"], T, c["parent"].data_ptr(), c["d_state"].data_ptr(), c["d_conv"].data_ptr(),
                  c["d_slot"].data_ptr(), c["N"], c["out"].data_ptr(), 0, c["stream"].cuda_stream) for c in cases]
    assert two_callers("gdn_decode_tree", *calls) == 0
    assert all(bool((c["out"] == 0).all()) for c in cases)


def test_two_threads_call_decode_tree_commit_with_different_sizes(two_callers):
    cases = [no_slots(160, 3, 6), no_slots(160, 3, 8)]
    calls = [Call(ctypes.addressof(c["s"]), c["N"], 3, c["parent"].data_ptr(), c["acc"].data_ptr(), c["d_state"].data_ptr(),
                  c["d_state"].data_ptr(), c["d_conv"].data_ptr(), c["d_conv"].data_ptr(), c["d_slot"].data_ptr(), c["N"], 0,
                  c["stream"].cuda_stream) for c in cases]
    assert two_callers("gdn_decode_tree_commit", *calls) == 0

def test_two_threads_call_decode_multi_with_different_sizes(two_callers):
    cases = [no_slots(160, 8, 6), no_slots(160, 8, 8)]
    calls = [Call(ctypes.addressof(c["s"]), c["N"], 8, c["d_state"].data_ptr(), c["d_conv"].data_ptr(), c["d_slot"].data_ptr(),
                  c["N"], c["out"].data_ptr(), 0, c["stream"].cuda_stream) for c in cases]
    assert two_callers("gdn_decode_multi", *calls) == 0


def test_two_threads_call_gemm_of_few_rows_with_different_sizes(two_callers):
    """A layer's two projections of up to 4 rows, as a tree of few nodes makes them, on two threads."""
    mats, calls = [], []
    for K in (64, 8192):
        a, b, out = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((4, K), (32, K), (4, 32)))
        mats.append((a, b, out, torch.cuda.Stream()))
        calls.append(Call(a.data_ptr(), K, b.data_ptr(), K, out.data_ptr(), 32, 4, 32, K, 0, mats[-1][3].cuda_stream))
    assert two_callers("gdn_gemm_bf16", *calls) == 0


# ------------------------------------------------------------------ bindings

def test_single_rows_of_any_stride():
    """One token: the stride of its (only) row means nothing."""
    D, H = 128, 2
    buf = torch.randn(H * D + 1, device="cuda").to(torch.bfloat16)
    x = buf.as_strided((1, H, D), (H * D + 1, D, 1))
    rope = gdn.make_rope(D)
    want = gdn.qk_norm_rope(rope, x.contiguous(), x.contiguous(), x.contiguous())
    got = gdn.qk_norm_rope(rope, x, x, x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c = attn_case(1, 1, 2, 1, D, [70], "chain", seed=91)
    want = attn_run(c)
    odd = {}
    for k in ("q", "kt", "vt", "g"):
        h = c[k].shape[1]
        odd[k] = torch.empty(h * D + 1, dtype=torch.bfloat16, device="cuda").as_strided((1, h, D), (h * D + 1, D, 1))
        odd[k].copy_(c[k])
    assert torch.equal(attn_run(c | odd), want)


def test_attention_tree_of_no_sequences():
    """A batch of no sequences, with and without a tree: no rows."""
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    for parent in (None, torch.empty(0, 5, dtype=torch.int32, device="cuda")):
        out = gdn.attention_tree(e(0, 4, 128), e(0, 2, 128), e(0, 2, 128), e(0, 9, 2, 128), e(0, 9, 2, 128),
                                 torch.empty(0, dtype=torch.int32, device="cuda"), parent)
        assert out.shape == (0, 512)


# ------------------------------------------------------------------ layers

@pytest.mark.parametrize("N,T", [(1, 1), (1, 3), (2, 11), (3, 40), (160, 5)])
def test_layer_tree_calls_are_their_parts(N, T):
    """Both layers' tree calls: bitwise the projection, the direct calls on its columns and the other projection; the commits
    those of the direct calls on what the workspace keeps."""
    g = torch.Generator().manual_seed(N + T)
    hidden, H_k, H_v, cap = 192, 2, 6, 90

    def mat(r, c):
        return (torch.randn(r, c, generator=g) * c ** -0.5).to(torch.bfloat16).cuda()

    rows = make_tree("holes", N, T, seed=N)
    parent = dev_tree(rows)
    ps = [oracle.tree.paths(r) for r in rows]
    acc = torch.tensor([max((t for t in range(T) if p[t]), key=lambda t: len(p[t])) for p in ps], dtype=torch.int32, device="cuda")
    x = torch.randn(N * T, hidden, generator=g).to(torch.bfloat16).cuda()
    # the delta-rule layer
    n_in = int(gdn.load().gdn_layer_n_in(H_k, H_v))
    w_in, w_out = mat(n_in, hidden), mat(hidden, H_v * 128)
    conv_w = (torch.randn((2 * H_k + H_v) * 128, 4, generator=g) * 0.5).to(torch.bfloat16).cuda()
    A_log = (torch.rand(H_v, generator=g) * 2).cuda()
    norm_w = (1 + 0.1 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda()
    L = gdn.make_layer(w_in, w_out, conv_w, A_log, norm_w, H_k, H_v, scale=0.7)
    S = (torch.randn(N, H_v, 128, 128, generator=g) * 0.1).cuda()
    C = torch.randn(N, 3, (2 * H_k + H_v) * 128, generator=g).to(torch.bfloat16).cuda()
    ws = gdn.layer_tree_workspace(L, N, T, "cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = gdn.layer_decode_tree(L, N, T, parent, x, S, C, ws, err=err)
    proj = torch.empty(N * T, -(-n_in // 8) * 8, dtype=torch.bfloat16, device="cuda")
    gdn.gemm_bf16(x, w_in, out=proj[:, :n_in])
    q, k, v, z, a, b = proj[:, :n_in].split([H_k * 128, H_k * 128, H_v * 128, H_v * 128, H_v, H_v], 1)
    s = gdn.make_inputs(q, k, v, a, b, z, conv_w, A_log, norm_w, scale=0.7)
    assert torch.equal(gdn.gemm_bf16(gdn.decode_tree(s, N, T, parent, S, C).view(N * T, -1), w_out), y)
    S2, C2 = gdn.decode_tree_commit(s, N, T, parent, acc, S, C, state_out=torch.empty_like(S), conv_out=torch.empty_like(C))
    gdn.layer_tree_commit(L, N, T, parent, acc, S, C, ws, err=err)
    assert torch.equal(S, S2) and torch.equal(C, C2)
    # the attention layer, on the other's output
    w_in, w_out = mat(gdn.ATTN_N_IN, hidden), mat(hidden, 24 * 256)
    nq, nk = ((1 + 0.1 * torch.randn(256, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    L = gdn.make_attn_layer(w_in, w_out, nq, nk)
    kc, vc = (torch.randn(N, cap, 4, 256, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    lens = torch.tensor([(n * 7) % (cap - T + 1) for n in range(N)], dtype=torch.int32, device="cuda")
    ws = gdn.attn_layer_tree_workspace(N, T, "cuda")
    x = y
    y = gdn.attn_layer_decode_tree(L, N, T, parent, x, kc, vc, lens, ws, err=err)
    q, gate, k, v = gdn.gemm_bf16(x, w_in).split([24 * 256, 24 * 256, 4 * 256, 4 * 256], 1)
    heads = lambda t: t.unflatten(1, (-1, 256))
    depth = torch.tensor([[max(len(p) - 1, 0) for p in tree] for tree in ps], dtype=torch.int32, device="cuda")
    pos = (lens[:, None] + depth).reshape(-1)
    q, k, _ = gdn.qk_norm_rope(gdn.make_rope(256, 64), heads(q), heads(k), q_norm_w=nq, k_norm_w=nk, positions=pos)
    there = torch.tensor([bool(p) for tree in ps for p in tree], device="cuda")
    out = gdn.attention_tree(q, k, heads(v), kc, vc, lens, parent, g=heads(gate))
    assert torch.equal(gdn.gemm_bf16(out, w_out), y) and bool((y[~there] == 0).all())
    kc2, vc2, lens2 = kc.clone(), vc.clone(), lens.clone()
    gdn.attn_tree_commit(k, heads(v), T, parent, acc, kc2, vc2, lens2)
    gdn.attn_layer_tree_commit(N, T, parent, acc, kc, vc, lens, ws, err=err)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and torch.equal(lens, lens2)
    assert int(err.item()) == 0
