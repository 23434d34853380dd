"""Host-side tests of what the rotation, norm and draft-tree calls do with what they cannot use: notes
that were never written, truth values that raise, sizes that do not fit, tensors that overlap (no GPU)."""
import os
import struct
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_memory_b200", "csrc")

NOTES = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include "tree_notes.h"

// The merge's loads and stores for a note, as tree_combine_kernel makes them: parts slot by slot,
// output rows of a block of up to `nt` row tiles of `tt` drafts.
static bool inside(const msa::MergeNote& n, int B, int M, int n_kv, int G, int tt, int nt, int ctas) {
  if (n.last - (int64_t)n.first > ctas) return false;  // the loop over the parts ends
  for (int64_t c = n.first; c <= n.last; ++c) {
    const int64_t slot = c > n.first ? 2 * (c * n_kv + n.head) : n.slot;
    if (slot < 0 || slot >= 2 * ctas) return false;
  }
  const int64_t rows = (int64_t)B * M * n_kv * G;
  for (int64_t i = 0; i < (int64_t)nt * tt; ++i) {
    const int64_t t = n.draft + i;
    if (t >= M) break;  // the kernel returns
    for (int g = 0; g < G; ++g) {
      const int64_t row = ((int64_t)n.query * M + t) * n_kv * G + (int64_t)n.head * G + g;
      if (t < 0 || row < 0 || row >= rows) return false;
    }
  }
  return true;
}

int main() {
  std::mt19937 rng(7);
  const int sizes[][4] = {{1, 1, 1, 1}, {8, 16, 8, 4}, {8, 200, 8, 4}, {4096, 256, 1, 16}, {33, 5, 3, 7}, {2, 255, 7, 2}};
  long passed = 0, real = 0;
  for (auto& s : sizes)
    for (int ctas : {8, 132, 148}) {
      const int B = s[0], M = s[1], n_kv = s[2], G = s[3], tt = 128 / G, nt = M > tt ? 2 : 1, groups = ctas / n_kv;
      auto note = [&](const int32_t (&v)[7]) { return msa::MergeNote{v[0], v[1], v[2], v[3], v[4], v[5], v[6]}; };
      auto ok = [&](const msa::MergeNote& n) { return msa::merge_note_ok(n, B, M, n_kv, groups); };
      const int32_t edge[] = {0, 1, -1, 2, B - 1, B, M - 1, M, n_kv - 1, n_kv, groups - 1, groups, ctas, 2 * ctas - 1, 2 * ctas,
                              INT32_MAX, INT32_MIN, 0x7F7F7F7F, (int32_t)0xFEFEFEFE, 1 << 30};
      for (int it = 0; it < 300000; ++it) {
        int32_t v[7];
        for (int32_t& x : v) x = rng() % 3 == 0 ? (int32_t)rng() : edge[rng() % (sizeof(edge) / sizeof(edge[0]))];
        if (rng() % 4 == 0) v[6] = 2 * (int32_t)((uint32_t)v[4] * (uint32_t)n_kv + (uint32_t)v[2]) + (int)(rng() % 2);
        if (!ok(note(v))) continue;
        ++passed;
        if (!inside(note(v), B, M, n_kv, G, tt, nt, ctas)) {
          printf("a note outside its buffers passed: %d %d %d %d %d %d %d\n", v[0], v[1], v[2], v[3], v[4], v[5], v[6]);
          return 1;
        }
      }
      for (int c = 0; c + 1 < groups; ++c)  // what the kernel writes for a cut item
        for (int h = 0; h < n_kv; ++h)
          for (int last = c + 1; last < groups; ++last)
            for (int second = 0; second < 2; ++second, ++real)
              if (!ok({B - 1, (M - 1) / (nt * tt) * nt * tt, h, M, c, last, 2 * (c * n_kv + h) + second}) || ok({-1, 0, h, M, c, last, 2 * (c * n_kv + h)})) {
                printf("a real note was refused\n");
                return 1;
              }
    }
  printf("%ld %ld\n", passed, real);
  return passed > 100 && real > 1000 ? 0 : 1;
}
"""


def test_merge_notes_that_nobody_wrote_stay_inside_their_buffers(tmp_path):
    """The merge of a draft-tree attention after a CTA gave up waiting: whatever the workspace held in the
    place of its note, a note that the merge takes indexes nothing outside the parts and the output."""
    src, exe = tmp_path / "notes.cpp", tmp_path / "notes"
    src.write_text(NOTES)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    # and the kernel asks before it uses one
    text = open(os.path.join(CSRC, "tree.cu"), encoding="utf-8").read()
    merge = text[text.index("tree_combine_kernel(const"):text.index("// drafts per row tile")]
    assert merge.index("merge_note_ok(") < min(merge.index("p.part_ml"), merge.index("p.out +"))


@pytest.fixture(scope="module")
def msa():
    from long_context_memory_b200 import build

    if build.needs_build():
        build.build()
    import long_context_memory_b200 as m

    return m


def test_a_truth_value_that_raises_is_passed_on(msa):
    """rotate's ``grad`` is read before anything is launched, and its error is the caller's."""
    import torch

    q, pos = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="ambiguous"):
        msa.rotate(msa.rotary(64), q, pos, grad=torch.zeros(2))


def test_heads_beyond_32_bits_are_refused(msa):
    """2^32 + 1 heads (of a broadcast tensor) are not one head."""
    import torch

    q = torch.zeros(1, 1, 64).expand(1, 2 ** 32 + 1, 64)
    out = torch.zeros(1, 1, 64).expand(1, 2 ** 32 + 1, 64)
    pos = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="heads"):
        msa.rotate(msa.rotary(64), q, pos, out=out)
    with pytest.raises(ValueError, match="heads"):
        msa.head_norm_rotate(msa.rotary(64), q, None, None, None, pos, out=out)
    with pytest.raises(ValueError, match="CUDA"):  # what fits is told that it wants CUDA tensors
        msa.rotate(msa.rotary(64), q[:, :3], pos)


SHARE = r"""
#include <cstdio>
#include <random>
#include <set>
#include <vector>
#include "overlap.h"
using msa::Blocks;
static std::vector<char> bytes(const Blocks& t) {
  std::vector<char> v(6000, 0);
  for (int r = 0; r < t.rows; ++r)
    for (int h = 0; h < t.heads; ++h)
      for (int e = 0; e < t.width; ++e) v[t.base + r * t.row + h * t.head + e] = 1;
  return v;
}
int main() {
  std::mt19937 rng(11);
  auto u = [&](int n) { return (int64_t)(rng() % n); };
  long shared = 0, apart = 0, careful = 0;
  for (int it = 0; it < 200000; ++it) {
    Blocks a, b;
    const int64_t pitch = 1 + u(60), head = 1 + u(30);
    for (Blocks* t : {&a, &b}) {
      *t = {(uintptr_t)u(400), 1 + u(6), 1 + u(6), u(4) ? pitch * (1 + (u(3) == 0)) : u(120), u(4) ? head : u(60), 1 + u(12)};
      if (u(8) == 0) std::swap(t->row, t->head);
    }
    const std::vector<char> va = bytes(a), vb = bytes(b);
    bool truth = false;
    for (size_t i = 0; i < va.size(); ++i) truth |= va[i] && vb[i];
    const bool got = msa::share_bytes(a, b);
    if (got != msa::share_bytes(b, a)) return printf("not symmetric\n"), 1;
    if (truth && !got) return printf("a shared byte was missed\n"), 1;
    auto one = [](int64_t n, int64_t s, int64_t m, int64_t t) { return n == 1 || s == 0 || m == 1 || t == 0 || s == t; };
    const bool exact = one(a.rows, a.row, b.rows, b.row) || one(a.heads, a.head, b.heads, b.head);
    if (exact && got != truth) return printf("tensors apart were taken for sharing\n"), 1;
    ++(truth ? shared : got ? careful : apart);
  }
  // sizes of real calls: slices of a fused projection, head-major and interleaved heads, far rows
  auto T = [](int64_t base, int64_t rows, int64_t heads, int64_t row, int64_t head, int64_t width) { return Blocks{(uintptr_t)base, rows, heads, row, head, width}; };
  const int64_t W = 256, R = 48 * W, N = 1 << 30;
  struct { Blocks a, b; bool share; } real[] = {
      {T(0, N, 32, R, W, W), T(32 * W, N, 8, R, W, W), false},         // q and k of one projection
      {T(0, N, 32, R, W, W), T(32 * W - 2, N, 8, R, W, W), true},
      {T(R, N, 32, R, W, W), T(40 * W, N, 8, R, W, W), false},
      {T(0, N, 32, R, W, W), T(R, N, 32, R, W, W), true},              // one row off
      {T(0, N, 16, 48 * W, 3 * W, W), T(W, N, 16, 48 * W, 3 * W, W), false},  // q, k, v of a head side by side
      {T(0, N, 16, 48 * W, 3 * W, W), T(2 * W + 2, N, 16, 48 * W, 3 * W, W), true},
      {T(0, N, 32, W, N * W, W), T(32 * N * W, N, 8, W, N * W, W), false},    // head-major
      {T(0, N, 32, W, N * W, W), T(31 * N * W, N, 8, W, N * W, W), true},
      {T(0, 1, 32, 7, W, W), T(16 * W, N, 1, R, 9, W), true},
      {T(1 << 20, INT64_C(2147483647), 65535, INT64_MAX, INT64_MAX, W), T(0, 1, 1, 0, 0, 1 << 20), false},
      {T(0, 0, 4, R, W, W), T(0, 3, 4, R, W, W), false}};
  for (auto& c : real)
    if (msa::share_bytes(c.a, c.b) != c.share || msa::share_bytes(c.b, c.a) != c.share) return printf("case %ld\n", (long)(&c - real)), 1;
  printf("%ld %ld %ld\n", shared, apart, careful);
  return shared > 1000 && apart > 1000 ? 0 : 1;
}
"""


def test_share_bytes_against_enumeration(tmp_path):
    """The overlap check of two strided tensors against their bytes, one by one."""
    src, exe = tmp_path / "share.cpp", tmp_path / "share"
    src.write_text(SHARE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


FAKE = 0x100000  # 16-byte aligned non-null "device" address; never dereferenced


def _heads(heads, D, inp, out, in_row, in_head, out_row, out_head):
    return struct.pack("@PPqqqqii", inp, out, in_row, in_head, out_row, out_head, heads, 0)


@pytest.mark.parametrize("form", ["rotate", "forward", "backward"])
@pytest.mark.parametrize("dtype,size", [(0, 2), (2, 4)])
def test_an_output_that_overlaps_its_input_is_refused(msa, monkeypatch, form, dtype, size):
    """In place, or apart: an output some rows, heads or elements off its input would be read after it was
    written.  Outputs that interleave with their input share nothing and are taken."""
    monkeypatch.setenv("MSA_FAULT", "launch")  # valid calls stop with MSA_ERR_CUDA before their first launch
    import ctypes

    D, heads, rows = 64, 4, 10
    r, far = msa.rotary(D), FAKE + (1 << 40)

    def call(off, strides_in, strides_out):
        h = _heads(heads, D, FAKE, FAKE + off * size, *strides_in, *strides_out)
        if form == "rotate":
            return msa.lib.msa_rotate(ctypes.byref(r), dtype, h, None, rows, far, 0, None)
        if form == "forward":
            return msa.lib.msa_head_norm_rotate(ctypes.byref(r), dtype, h, None, rows, None, None, 0.0, 1e-6, far, None)
        x = _heads(heads, D, far, far, *strides_in, *strides_in)
        return msa.lib.msa_head_norm_rotate_grad(ctypes.byref(r), dtype, x, None, h, None, rows, None, None, 0.0, 1e-6, far,
                                                 None, None, far, 1 << 24, None)

    flat, wide = (heads * D, D), (2 * heads * D, D)
    for off in (0, rows * heads * D, 1 << 30):  # in place; right behind; far away
        assert call(off, flat, flat) == 4
    for off in (1, 8, D, heads * D, 3 * heads * D, rows * heads * D - 1):
        assert call(off, flat, flat) == 1, off
    assert call(0, flat, wide) == 1                    # in place with another pitch
    assert call(0, (D, rows * D), flat) == 1           # in place, the heads' order turned round
    assert call(heads * D, wide, wide) == 4            # the other half of every row
    assert call(heads * D - 1, wide, wide) == 1
    assert call(heads * D + 1, wide, wide) == 1
    assert call(D, (8 * D, 2 * D), (8 * D, 2 * D)) == 4  # heads side by side
    assert call(0, (0, 0), flat) == 1                  # a broadcast input inside its output
    assert call(heads * D, (0, 0), flat) == 4


def test_the_binding_refuses_outputs_inside_other_tensors(msa):
    """Outputs that share memory with another output or input of the call.  (Host tensors: what fits is told
    that it wants CUDA tensors.)"""
    import torch

    def fits(f, *a, **kw):
        with pytest.raises(ValueError, match="CUDA"):
            f(*a, **kw)

    def clash(f, *a, **kw):
        with pytest.raises(ValueError, match="overlap"):
            f(*a, **kw)

    R, D, r = 6, 64, msa.rotary(64)
    fused = torch.zeros(R, 12, D)  # 8 query, 2 key, 2 value heads of one projection
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    pos, slots = torch.zeros(R, dtype=torch.int32), torch.zeros(R, dtype=torch.int32)
    w = torch.ones(D)
    new = torch.empty_like
    for f, a in ((msa.rotate, (r, q, pos)), (lambda *x, k, **kw: msa.head_norm_rotate(x[0], x[1], k, w, w, x[2], **kw), (r, q, pos))):
        fits(f, *a, k=k, out=q, k_out=k)                  # both in place
        fits(f, *a, k=k, out=new(q), k_out=new(k))
        fits(f, *a, k=fused[:, :2], out=new(q))           # inputs may share
        clash(f, *a, k=k, k_out=q[:, 2:4])                # the keys' output inside the queries
        clash(f, *a, k=k, out=fused[:, 4:])               # the queries' output over the keys
        o = torch.zeros(R, 8, D)
        clash(f, *a, k=k, out=o, k_out=o[:, 6:])
        clash(f, *a, k=k, out=o, k_out=o.view(-1)[D:D + R * 2 * D].view(R, 2, D))
        store = torch.zeros(R * 8 * D)                    # positions inside an output
        clash(f, r, q, store.view(torch.int32)[D:D + R], k=k, out=store.view(R, 8, D))
    clash(msa.head_norm_rotate, r, q, None, fused[2, 3], None, pos, out=q)  # a weight inside the output
    K, V = torch.zeros(2, 9, 2, D), torch.zeros(2, 9, 2, D)
    app = lambda q=q, k=k, v=v, K=K, V=V, w=w, pos=pos, slots=slots, **kw: msa.head_norm_append(r, q, k, v, w, w, pos, slots, K, V, **kw)
    fits(app, out=q)
    fits(app)
    clash(app, out=fused[:, 2:10])
    clash(app, out=fused[:, 4:])
    for name in ("K", "V"):
        cache = torch.zeros(2, 9, 2, D)
        rows = cache.view(18, 2, D)[:R]
        wide = cache.view(-1)[:R * 2 * D].view(R, 2, D)
        clash(app, **{name: cache}, k=rows)
        clash(app, **{name: cache}, v=rows)
        clash(app, **{name: cache}, q=wide)
        clash(app, **{name: cache}, q=wide, out=new(wide))
        clash(app, **{name: cache}, q=k, out=wide)
        clash(app, **{name: cache}, w=cache.view(-1)[64:128])
        clash(app, **{name: cache}, pos=cache.view(torch.int32).view(-1)[:R])
        clash(app, **{name: cache}, slots=cache.view(torch.int32).view(-1)[-R:])
    g = torch.zeros(R, 12, D)
    dq, dk = g[:, :8], g[:, 8:10]
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    W = lambda: torch.zeros(D)
    back = lambda out, w=w: msa.head_norm_rotate_grad(r, q, k, w, w, pos, dq, dk, out=out, ws=ws)
    fits(back, (new(q), new(k), W(), W()))
    fits(back, (dq, dk, W(), W()))                        # over the outputs' gradients
    fits(back, (q, k, None, None))                        # over the inputs
    clash(back, (fused[:, 1:9], new(k), W(), W()))
    clash(back, (new(q), dq[:, :2], W(), W()))
    clash(back, (new(q), q[:, :2], W(), W()))
    clash(back, (g[:, 4:], new(k), W(), W()))
    clash(back, (fused[:, 4:], new(k), W(), W()))
    o = torch.zeros(R, 8, D)
    clash(back, (o, o[:, :2], W(), W()))
    clash(back, (o, new(k), o[2, 3], W()))
    clash(back, (new(q), o[:, :2], W(), o[5, 1]))
    x = torch.zeros(2 * D)
    clash(back, (new(q), new(k), x[:D], x[1:D + 1]))
    clash(back, (o, new(k), None, None), w=o[1, 1])
    fits(back, (new(q), new(k), x[:D], x[D:]))


@pytest.fixture
def commands(monkeypatch):
    """The build's commands, recorded instead of run; those that name a word of ``fail`` fail."""
    from long_context_memory_b200 import build

    class Done:
        returncode, stdout, stderr = 0, "", ""

    seen, fail = [], []

    def run(cmd, **kw):
        seen.append(cmd)
        d = Done()
        d.returncode = int(any(w in str(c) for c in cmd for w in fail))
        return d

    monkeypatch.setattr(build.subprocess, "run", run)
    return build, seen, fail


def _linked(build, seen):
    return [i for i, c in enumerate(seen) if build.LIB in c]


def test_the_library_builds_without_pytorch(commands, monkeypatch, capsys):
    """libmsa.so needs nvcc alone: the C ABI's users need no PyTorch."""
    import sys

    build, seen, fail = commands
    for name in {"torch"} | {m for m in sys.modules if m.startswith("torch.")}:
        monkeypatch.setitem(sys.modules, name, None)
    assert build.build() == build.LIB
    assert len(_linked(build, seen)) == 1 and not any(build.FAST in c for c in seen)
    assert "_fastcall" in capsys.readouterr().err  # and it says what was left out
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(build, "FAST", build.FAST + ".missing")
    assert not build.needs_build()  # a library alone is up to date then


def test_the_library_is_linked_although_the_binding_s_part_fails(commands):
    build, seen, fail = commands
    fail.append("fastcall.cpp")
    with pytest.raises(RuntimeError, match="_fastcall"):
        build.build()
    assert len(_linked(build, seen)) == 1
    fail[:] = ["tree.cu"]
    with pytest.raises(RuntimeError, match="libmsa"):
        build.build()


def test_the_tree_attention_s_output_stays_off_its_small_inputs(msa, monkeypatch):
    """out over the mask, the lengths, the documents or the routing: other CTAs would read what was written."""
    import ctypes

    monkeypatch.setenv("MSA_FAULT", "launch")
    d = msa.Dims(64, 8, 2, 64, 1, 64, 64, 1e6)
    B, M, T, k, n_docs, n_chunks = 2, 40, 10, 3, 50, 90
    need = msa.lib.msa_tree_attend_workspace_size(ctypes.byref(d), B, M, k, T)
    far = FAKE + (1 << 40)

    def call(out=far, mask=FAKE, n_draft=None, loc=FAKE, off=FAKE, top=FAKE):
        return msa.lib.msa_tree_attend(ctypes.byref(d), FAKE, FAKE, FAKE, mask, n_draft, B, M, FAKE, FAKE, loc, T, FAKE, FAKE, off,
                                       n_docs, n_chunks, top, k, 0.0, out, FAKE, need, None)

    size = B * M * 8 * 64 * 2
    assert call() == 4
    for name, n in (("mask", B * M * 2 * 4), ("n_draft", B * 4), ("loc", B * 4), ("off", (n_docs + 1) * 4), ("top", B * k * 4)):
        assert call(**{name: far + size}) == 4, name          # right behind
        assert call(**{name: far + size - 16}) == 1, name
        assert call(**{name: far - (n + 15) // 16 * 16}) == 4, name
        assert call(**{name: far - n // 16 * 16 + (0 if n % 16 else 16)}) == 1, name
