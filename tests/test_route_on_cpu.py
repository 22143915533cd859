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

# The exponential as CUDA's may be: within two steps of the result's last place of the exact value, where `salt` says (0: nearest).
EXP = """
static unsigned salt;
static float expf_on_gpu(float x) {
  const double exact = exp((double)x);
  float v = (float)exact;
  if (!salt || !std::isfinite(v) || v == 0.0f) return v;
  uint32_t bits;
  std::memcpy(&bits, &x, 4);
  bits = (bits ^ salt) * 2654435761u;
  bits = (bits ^ bits >> 15) * 2246822519u;
  const float to = bits & 0x100 ? INFINITY : 0.0f;
  const double step = std::fabs((double)std::nextafterf(v, INFINITY) - v);
  for (int i = 0; i < 2; ++i) {
    const float w = std::nextafterf(v, to);
    if (std::isfinite(w) && std::fabs(w - exact) <= 2 * step) v = w;
  }
  return v;
}
#define expf expf_on_gpu
"""

ENTRY = """
extern "C" void set_salt(unsigned s) { salt = s; }
extern "C" float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }
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
        f.write('#include "warp_on_cpu.h"\n' + EXP + 'static std::vector<double> shared;\nstatic int experts;\nnamespace mx {\nnamespace swiglu_math {\n'
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
    """Experts equal, unless c or two groups' values differ by no more than double precision rounds a score and a bias by."""
    ids, _ = _run(lib, logits, k, score, bias, groups, top)
    l, c = _c(logits, score, bias)
    # two steps of the last place for a score, half of one for the sum
    off = 2.5 * 2.0 ** -52 * (np.where(np.isneginf(l), 0, _c(logits, score, None)[1]) + (0 if bias is None else np.abs(np.asarray(bias, np.float64))))
    size = l.shape[1] // groups
    for t in range(len(l)):
        allowed = range(l.shape[1])
        if top < groups:
            with np.errstate(invalid="ignore"):
                worth = np.sort(c[t].reshape(groups, -1), 1)[:, ::-1][:, :2].sum(1)
            order = sorted(range(groups), key=lambda g: (-worth[g], g))
            a, b = order[top - 1], order[top]
            both = [e for e in allowed if e // size in (a, b)]
            with np.errstate(invalid="ignore"):
                if np.isnan(worth).any() or (worth[a] != worth[b] and worth[a] < worth[b] + 2 * off[t, both].max()):
                    continue
            allowed = [e for e in allowed if e // size in order[:top]]
        key = l[t] if bias is None else c[t]
        want = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        if ids[t].tolist() != want:
            x, y = key[ids[t]], key[want]
            with np.errstate(invalid="ignore"):
                near = (x == y) | (np.abs(x - y) <= off[t, ids[t]] + off[t, want])
            assert near.all() and (x != y).any(), (t, ids[t].tolist(), want, x, y)


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
    try:
        for seed in range(part * 40, part * 40 + 40):
            lib.set_salt(seed)
            _check(lib, *_random(seed))
    finally:
        lib.set_salt(0)


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


@pytest.mark.parametrize("salt", [1, 5, 12])
@pytest.mark.parametrize("binade", [1, 3, 6, 10])
def test_scores_as_far_off_as_documented(lib, salt, binade):
    """CUDA documents two steps of the last place for expf.  Of two experts, one whose fp32 score is too large by as much as
    there is among many logits and one whose score is as much too small, with biases that leave the second a little more:
    fp32 puts the first ahead, by nearly what its scores may be off together."""
    lib.sigmoid.restype = ctypes.c_float
    x = -np.float32(np.log(2)) * binade - np.random.default_rng(binade).random(20000).astype(np.float32) * np.float32(0.02)
    x = np.float32(np.where(binade == 1, -x, x))     # scores above a half too
    try:
        lib.set_salt(salt)
        got = np.array([lib.sigmoid(ctypes.c_float(v)) for v in x], np.float64)
        exact = 1 / (1 + np.exp(-x.astype(np.float64)))
        order = np.argsort((got - exact) / exact)
        low, high = order[:40], order[-40:]
        bias = (-exact).astype(np.float32)
        left = exact + bias.astype(np.float64)
        step = np.spacing(bias[low[0]]).astype(np.float64)
        for i in high:
            ahead = (left[i] - left[low]) % abs(step)          # what the other's bias, in whole steps, leaves to go
            j = low[np.argmax(ahead)]
            b = np.float32(bias[j].astype(np.float64) + np.ceil((left[i] - left[j]) / abs(step)) * abs(step))
            for first, second in ((i, j), (j, i)):
                bb = np.array([bias[i], b] if first == i else [b, bias[i]] , np.float32)
                l = np.array([[x[first], x[second], -50.0]])
                for k in (1, 2):
                    _check(lib, l, k, "sigmoid", np.r_[bb, np.float32(-9)])
    finally:
        lib.set_salt(0)


@pytest.mark.parametrize("far", [88.8, 89.5, 95.0, 100.0])
def test_scores_that_underflow_beside_biases_as_small(lib, far):
    """Sigmoid scores of some 2^-128, which fp32 has as 0 where e^-x overflows, against biases of that size."""
    for n in range(1, 40):
        l = np.array([[-101.0, -far, 0.0, 0.0]])
        _check(lib, l, 2, "sigmoid", np.array([n * 2.0 ** -133, 0.0, -3.0, -3.0], np.float32))
        _check(lib, l, 1, "sigmoid", np.array([n * 2.0 ** -133, 0.0, -3.0, -3.0], np.float32))
