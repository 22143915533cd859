"""The router's kernel, its own source, on the host: a warp's lanes one after the other, every index that it works out from
its data checked, and the experts against those of c in double precision.  Its inputs are those that its fp32 scores, and
those of 44 bits, leave open: near-ties, twins, infinities, and logits at the ends of the exponential's range."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "block_scaled_mlp_gb300", "csrc")

ENTRY = """
static mx::RouteParams params;
static int width, score;
template <int V>
static void kernel() { score ? mx::moe_route_kernel<V, true, true>(params) : mx::moe_route_kernel<V, true, false>(params); }
static void one_lane() {
  switch (width) {
    case 1: return kernel<1>();
    case 2: return kernel<2>();
    case 4: return kernel<4>();
    case 8: return kernel<8>();
    default: return kernel<32>();
  }
}
// Tokens one after the other; the number of them in which an index was out of its bounds.
extern "C" long route(const float* logits, long T, int E, int k, int sigmoid, float* bias, int groups, int top, int renorm, int* ids,
                      float* weights, char* what) {
  long bad = 0;
  shared.assign(mx::ROUTE_WARPS * E, 0.0);
  experts = E;
  for (width = 1; 32 * width < E;) width *= 2;
  score = sigmoid;
  for (long t = 0; t < T; ++t) {
    params = mx::RouteParams{};
    params.logits = logits + t * E;
    params.bias = {bias, E, "bias"};
    params.ids = {ids + t * k, k, "ids"};
    params.weights = {weights + t * k, k, "weights"};
    params.T = 1; params.E = E; params.k = k; params.groups = top == groups ? 1 : groups; params.top_groups = top;
    params.wide = 1; params.sigmoid = sigmoid; params.renorm = renorm; params.scale = 1.0f;
    warp::faults = 0;
    warp::run(one_lane);
    if (warp::faults && !bad++) std::snprintf(what, 256, "token %ld: %s", t, warp::first_fault);
  }
  return bad;
}
"""


def _between(text, first, last):
    a = text.index(first)
    return text[a:text.index(last, a)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    math = _between(open(os.path.join(CSRC, "swiglu_math.cuh")).read(), "// ---- float-float", "// e^x as float-float")
    src = _between(open(os.path.join(CSRC, "route.cu")).read(), "constexpr uint32_t FULL", "struct RouteBwdParams")
    for old, new in (("const float* bias;", "warp::Checked<float> bias;"), ("int32_t* ids;", "warp::Checked<int32_t> ids;"),
                     ("float* weights;", "warp::Checked<float> weights;"), ("extern __shared__ double s_c[];", "double* s_c = shared.data();"),
                     ("bool wide, int e) {", "bool wide, int e) {\n  if (e < 0 || e >= experts) { warp::fault(\"logits\", e, experts); return 0; }"),
                     ("isinf(", "std::isinf(")):
        assert old in src, old
        src = src.replace(old, new)
    d = tmp_path_factory.mktemp("route")
    cpp, so = str(d / "route.cpp"), str(d / "route.so")
    with open(cpp, "w") as f:
        f.write('#include "warp_on_cpu.h"\nstatic std::vector<double> shared;\nstatic int experts;\nnamespace mx {\nnamespace swiglu_math {\n'
                "inline float rcp_approx(float x) { return 1.0f / x; }\n" + math + "}\nnamespace {\n" + src + "}\n}\n" + ENTRY)
    subprocess.run(["g++", "-std=c++20", "-O1", "-ffp-contract=off", "-w", "-fPIC", "-shared", "-I", os.path.join(TESTS, "probes"), cpp,
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.route.restype = ctypes.c_long
    return lib


def _run(lib, logits, k, score, bias=None, groups=1, top=1, renorm=True):
    l = np.ascontiguousarray(logits, np.float32)
    b = None if bias is None else np.ascontiguousarray(bias, np.float32)
    (T, E), what = l.shape, ctypes.create_string_buffer(256)
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k), np.float32)
    at = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)  # noqa: E731
    bad = lib.route(at(l), ctypes.c_long(T), E, k, score == "sigmoid", at(b), groups, top, renorm, at(ids), at(w), what)
    assert bad == 0, what.value.decode()
    return ids, w


def _c(logits, score, bias):
    l = np.asarray(logits, np.float32).astype(np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            m = l.max(1, keepdims=True)
            e = np.exp(l - np.where(np.isneginf(m), 0, m))
            s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
        return l, np.where(np.isneginf(l), -np.inf, s if bias is None else s + np.asarray(bias, np.float32).astype(np.float64))


def _check(lib, logits, k, score, bias=None, groups=1, top=1):
    """Experts equal, unless c or two groups' values differ by less than double precision's rounding of them."""
    ids, _ = _run(lib, logits, k, score, bias, groups, top)
    l, c = _c(logits, score, bias)
    size = l.shape[1] // groups
    for t in range(len(l)):
        allowed = range(l.shape[1])
        if top < groups:
            with np.errstate(invalid="ignore"):
                worth = np.sort(c[t].reshape(groups, -1), 1)[:, ::-1][:, :2].sum(1)
            order = sorted(range(groups), key=lambda g: (-worth[g], g))
            a, b = worth[order[top - 1]], worth[order[top]]
            if np.isnan(worth).any() or (a != b and a - b < 1e-15 * (1 + abs(a))):
                continue
            allowed = [e for e in allowed if e // size in order[:top]]
        key = l[t] if bias is None else c[t]
        want = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        if ids[t].tolist() != want:
            x, y = key[ids[t]], key[want]
            fine = np.isfinite(x) & np.isfinite(y)
            near = np.where(x == y, 0.0, 1.0)
            near[fine] = np.abs(x[fine] - y[fine]) / (1 + np.abs(x[fine]))
            assert 0 < near.max() < 4e-16, (t, ids[t].tolist(), want, x, y)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [88.4, 88.7, 89.0, 95.0, 140.0, 1e4])
def test_logits_beyond_the_range_of_44_bits(lib, score, far):
    """All experts of the groups that are taken are chosen, two of them are closer than fp32 can tell, and one has a logit
    that scores of 44 bits are not made for."""
    for groups, top, size in ((8, 3, 2), (31, 2, 3), (1, 1, 5), (4, 1, 9)):
        E = groups * size
        l = np.full((4, E), -30.0)
        l[:, :size * top] = 2.0 if score == "softmax" else 1.0
        for t in range(4):
            l[t, t % size] = 2.0 - far if score == "softmax" else -far
        s = _c(l, score, None)[1][0]
        bias = np.zeros(E, np.float32)
        bias[:size * top] = np.float32(0.5) - s[:size * top].astype(np.float32)
        bias[1:size * top:2] = np.nextafter(bias[1:size * top:2], np.float32(1))
        _check(lib, l, size * top, score, bias, groups, top)


def _random(seed):
    g = np.random.default_rng(seed)
    groups = int(g.choice([1, 1, 2, 3, 4, 8, 31, 32]))
    size = int(g.integers(1, max(2, 150 // groups + 1)))
    if seed % 40 == 0:
        size = 1024 // groups
    E, top, T = groups * size, int(g.integers(1, groups + 1)), 6
    most = min(32, top * size)
    k = most if g.random() < 0.4 else int(g.integers(1, most + 1))
    score = str(g.choice(["softmax", "sigmoid"]))
    special = [0.0, -0.0, 88.7, -88.7, -88.4, 64, -64, -64.5, -103, -150, 1e-20, 3e38, -3e38, 20, -20]
    l = g.normal(size=(T, E)) * g.choice([0.1, 1, 10, 40])
    at = g.random((T, E)) < g.choice([0, 0.1, 0.5, 1])
    l[at] = g.choice(special, int(at.sum()))
    l[g.integers(0, 4, T) == 1] = g.choice(special)
    l[g.random((T, E)) < g.choice([0, 0, 0.2, 0.8])] = -np.inf
    near = np.asarray(g.choice([0.7, 0, -0.3]) - np.where(np.isneginf(l), 0, _c(l, score, None)[1])[0], np.float32)
    for _ in range(2):
        near = np.where(g.random(E) < 0.4, np.nextafter(near, np.float32(np.inf)), near)
    bias = [None, g.choice([0, 1e-3, 2e-3], E), near, near, g.integers(0, 3, E) * 2.0 ** -float(g.integers(20, 100)) - 0.5,
            g.choice([0, 0.25, np.inf, -np.inf, 1e30], E, p=[0.4, 0.25, 0.05, 0.2, 0.1]), g.choice([0.0, -1.0, 2.0 ** -24], E)][g.integers(0, 7)]
    if bias is not None and g.random() < 0.15:
        e = int(g.integers(E))
        l[:, e], bias[e] = -np.inf, np.nan
    return l, k, score, bias, groups, top


@pytest.mark.filterwarnings("ignore:overflow")
@pytest.mark.parametrize("part", range(8))
def test_random_doubts(lib, part):
    for seed in range(part * 40, part * 40 + 40):
        l, k, score, bias, groups, top = _random(seed)
        _check(lib, l, k, score, bias, groups, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2, 3, 4, 8])
def test_group_values_past_the_largest_number(lib, score, size):
    """Experts put out of reach by the lowest finite bias, or ahead by the largest: a sum of two is none of fp32's numbers, and
    still ahead of minus infinity or behind plus infinity."""
    big = float(np.finfo(np.float32).max)
    for seed in range(40):
        g = np.random.default_rng(seed)
        groups = 4
        bias = g.choice([-big, -big, -3e38, 0.0, -np.inf] if seed % 2 else [big, 3e38, 0.0, np.inf, 0.25], groups * size)
        l = g.normal(size=(3, groups * size))
        l[1] = 0.5
        l[2, g.random(groups * size) < 0.3] = -np.inf
        _check(lib, l, int(g.integers(1, size + 1)), score, bias, groups, int(g.integers(1, groups)))
