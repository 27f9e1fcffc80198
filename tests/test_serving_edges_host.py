"""Serving operators without a GPU, beyond test_serving_host.py: rules that the
sources keep, and what the Python side and the build refuse or report."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SERVE = os.path.join(ROOT, "rank_biased_window_b200", "csrc", "serve")


def _functions(text):
    """(head, body) of every function of a source laid out with its braces in the first column."""
    for m in re.finditer(r"^((?:template|__global__|__device__|struct)[^;{}]*?\([^{};]*\)[^{};]*)\{\n(.*?)^\}",
                         text, re.M | re.S):
        yield m.group(1), m.group(2)


@pytest.mark.parametrize("name", ["rotary.cuh", "cache_append.cuh", "cache_attn.cuh", "cache_evict.cuh"])
def test_kernels_wait_before_they_read(name):
    """A kernel may start while the one before it runs, and only its wait makes
    earlier writes visible: it stands in the kernel itself, in front of whatever
    reads global memory, and on every way through it."""
    with open(os.path.join(SERVE, name)) as f:
        text = f.read()
    kernels = [(h, b) for h, b in _functions(text) if "__global__" in h]
    assert len(kernels) == text.count("__global__ ")
    for head, body in _functions(text):
        if "__global__" not in head:
            assert "grid_dep_wait" not in body, head
            continue
        assert body.count("grid_dep_wait()") == 1, head
        before = re.sub(r"//.*", "", body.split("grid_dep_wait()")[0])
        assert "return" not in before, head
        for read in ("__ld", "parts_of", "place_of", "segment_of", "select_begin", "a.lengths", "a.mass",
                     "a.kept", "a.pos[", "a.start[", "_mass<", "fetch", "bulk_load"):
            assert read not in before, (head, read)


WALK = r"""
#include "serve/cache_evict.cuh"
#include <cstdio>
int main() {
  rfb::EvictArgs a = {};
  int bad = 0;
  for (int heads : {1, 3, 64})
    for (int per_head : {1, 5, 33})
      for (int z0 : {0, 2})
        for (long long warps : {1, 8, 1184}) {
          a.heads = heads;
          const long long items = (long long)heads * per_head * (z0 == 0 ? 2 : 1);
          for (long long first = 0; first < warps; first += 7) {
            const int rounds = first < items ? (int)((items - first + warps - 1) / warps) : 0;
            const rfb::MoveWalk<false> w{a, z0, 0, first, warps, items, rounds, per_head};
            for (int round = 0; round < rounds + rfb::kMoveStages; ++round) {
              const auto p = w.at(round);
              bad += p.z < z0 || p.z > (z0 == 0 ? 1 : 2) || p.bh < 0 || p.bh >= heads ||
                     p.block < 0 || p.block >= per_head;
            }
          }
        }
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


def test_eviction_walk_names_only_what_exists(tmp_path):
    """The move's warps look up to two rounds past their last item: tensor, head and
    block have to exist there too."""
    import subprocess
    from rank_biased_window_b200 import build
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(WALK)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC,
                    "-o", str(exe), str(src)], check=True, capture_output=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "0\n"


def test_attention_with_counts_host_checks(rfb_lib):
    """The padded form checks as the plain one does, and has the plain one's arguments but one."""
    lib = rfb_lib.load_library()

    def call(B=1, H=2, Hk=1, Nq=1, cap=64, d=64, r=0, scale=0.1):
        return lib.rfb_attn_fwd_cache_counts(*([None] * 12), 1.0, None, None, None, 0, B, H, Hk, Nq,
                                             cap, d, r, scale, 1, None)
    assert call(B=0) == 0 and call(Nq=0) == 0 and call(H=0) == 0
    assert call() == 1 and call(scale=0.0) == 1 and call(H=3, Hk=2) == 1
    assert call(d=96) == 2 and call(r=12) == 2 and call(cap=33) == 2
    from rank_biased_window_b200.binding import SIGNATURES
    plain, padded = (SIGNATURES["rfb_attn_fwd_cache" + s][1] for s in ("", "_counts"))
    assert plain == padded[:9] + padded[10:]


def _host_cache(bind):
    c = [torch.zeros(2, 2, 64, ch, dtype=torch.uint8).view(torch.float8_e4m3fn) for ch in (64, 64, 8)]
    s = [torch.ones(2, 2, 2) for _ in range(3)]
    return bind.cache(*c, *s), c + s


@pytest.mark.parametrize("part", ["k", "v", "w", "k_scale", "v_scale", "w_scale"])
def test_cache_tensors_cannot_be_exchanged(part):
    """The calls hold the tensors that a cache was made of: another one in an attribute's
    place would be read by some of them only."""
    from rank_biased_window_b200 import Cache8
    c = object.__new__(Cache8)
    for name in (part, "cap", "device"):
        with pytest.raises(AttributeError, match="make a new Cache8"):
            setattr(c, name, torch.zeros(1))
    c.mass = None                   # looked at in each call


@pytest.mark.parametrize("change", [
    lambda t: t.resize_(2, 2, *[max(1, n // 2) for n in t.shape[2:]]),
    lambda t: t.set_(torch.zeros(1, dtype=t.dtype).expand(t.shape)),
    lambda t: setattr(t, "data", t.transpose(0, 1)),
    lambda t: setattr(t, "data", t.double().to(torch.float16)),
    lambda t: t.untyped_storage().resize_(0)])
@pytest.mark.parametrize("part", range(6))
def test_changed_cache_tensors_are_refused(rfb_lib, part, change):
    """A held tensor that was resized, freed or pointed elsewhere in place: its sizes are
    the cache's no longer, so no call may run with them."""
    from rank_biased_window_b200 import serving
    bind = serving._load_bind()
    held, tensors = _host_cache(bind)
    q = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    change(tensors[part])
    name = ("k", "v", "w", "k_scale", "v_scale", "w_scale")[part]
    for call in (lambda: bind.attn(held, q, q[..., :8], n, None, True, None, None, 1.0, None, None, None),
                 lambda: bind.append(held, None, q, q, q[..., :8], n, None),
                 lambda: bind.evict(held, None, held, None, n, 8, 0)):
        with pytest.raises(ValueError, match=f"the cache's {name} is not what it was"):
            call()


def test_written_memory_is_apart(rfb_lib):
    """What a call writes lies in nothing that it reads or writes besides, in whatever role;
    refused before any launch."""
    from rank_biased_window_b200 import serving
    bind = serving._load_bind()
    held, (k, v, w, ks, vs, ws) = _host_cache(bind)
    q, u = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 3, 8, dtype=torch.bfloat16)
    n, cnt = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    mass = torch.zeros(2, 2, 64)
    room = torch.zeros(1 << 16, dtype=torch.uint8)

    def part(dtype, shape, at=0):
        size = torch.empty(0, dtype=dtype).element_size() * torch.Size(shape).numel()
        return room[at: at + size].view(dtype).view(shape)

    def attn(**kw):
        a = dict(mass=None, mass_out=None, out=None, lse=None, workspace=None, counts=cnt)
        a.update(kw)
        return bind.attn(held, q, u, n, None, True, a["mass"], a["mass_out"], 1.0, a["out"], a["lse"],
                         a["workspace"], a["counts"])
    lse = part(torch.float32, (2, 4, 3))
    calls = [
        (lambda: attn(out=part(torch.bfloat16, q.shape), lse=lse), "lse .* out"),
        (lambda: attn(lse=lse, workspace=room), "workspace .* lse"),
        (lambda: attn(lse=lse, mass_out=part(torch.float32, mass.shape, 64)), "mass_out .* lse"),
        (lambda: attn(workspace=q), "workspace .* q"),
        (lambda: attn(workspace=u), "workspace .* u"),
        (lambda: attn(workspace=n), "workspace .* lengths"),
        (lambda: attn(workspace=cnt), "workspace .* counts"),
        (lambda: attn(workspace=mass, mass=mass, mass_out=mass), "workspace .* mass"),
        (lambda: attn(lse=ks.view(-1)[:0].new_zeros(2, 4, 3), workspace=vs), "workspace .* the cache's v_scale"),
        (lambda: attn(workspace=k), "workspace .* the cache's k"),
        (lambda: attn(out=q), "out .* q")]
    # a cache whose k and v exchange places, or that lies in one tensor twice
    swapped, twice = bind.cache(v, k, w, vs, ks, ws), bind.cache(k, k, w, ks, vs, ws)
    x = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16)
    new = torch.zeros(2, 2, 64)
    calls += [
        (lambda: bind.evict(held, mass, swapped, new, n, 8, 0), "out .* the cache"),
        (lambda: bind.evict(twice, mass, twice, mass, n, 8, 0), "the cache's v .* the cache's k"),
        (lambda: bind.append(twice, mass, x, x, x[..., :8], n, None), "the cache's v .* the cache's k"),
        (lambda: bind.append(held, k.view(-1)[: 4 * new.numel()].view(torch.float32).view(new.shape), x, x,
                             x[..., :8], n, None), "the cache's mass .* the cache's k")]
    for call, match in calls:
        with pytest.raises(ValueError, match=match.replace(" .* ", " must not share memory with ")):
            call()


@pytest.fixture
def elsewhere(rfb_lib, tmp_path, monkeypatch):
    """The build module with its products in a folder of their own."""
    import shutil
    from rank_biased_window_b200 import build
    for name in ("LIB", "BIND", "BIND_STAMP"):
        here = tmp_path / os.path.basename(getattr(build, name))
        shutil.copy2(getattr(build, name), here)
        monkeypatch.setattr(build, name, str(here))
    return build


def test_library_is_built_without_the_extension(elsewhere, monkeypatch, capsys):
    """Without a host compiler for the extension the library is built as ever, and no
    extension of other sources is left beside it."""
    made = []
    monkeypatch.setattr(elsewhere, "build_library", lambda *a: made.append(os.path.exists(elsewhere.BIND)))
    for cxx in ("/nonexistent/c++", "false"):
        monkeypatch.setenv("CXX", cxx)
        assert elsewhere.build(force=True) == elsewhere.LIB
        assert "is not" in capsys.readouterr().err and os.path.exists(elsewhere.BIND)
        with pytest.raises((RuntimeError, OSError)):
            elsewhere.build_bind(force=True)
    os.utime(elsewhere.BIND, (0, 0))
    assert elsewhere.build() == elsewhere.LIB
    assert "is not" in capsys.readouterr().err and not os.path.exists(elsewhere.BIND)
    assert made == [True] * 3       # the library came first


def test_extension_of_another_torch_is_built_again(elsewhere, monkeypatch):
    assert elsewhere.bind_up_to_date()
    monkeypatch.setenv("CXX", "false")
    assert elsewhere.build_bind() == elsewhere.BIND            # nothing to do
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert not elsewhere.bind_up_to_date()
    with pytest.raises(RuntimeError, match="failed"):
        elsewhere.build_bind()
    monkeypatch.undo()


def test_extension_shares_the_process_runtime(rfb_lib):
    """One C++ runtime in the process: the extension takes torch's, so that numbers go
    through its streams and torch's exceptions through its handlers (in a child, which a
    second runtime ends by a signal)."""
    import subprocess
    import sys
    code = """
import torch
from rank_biased_window_b200 import serving
bind = serving._load_bind()
c = torch.zeros(2, 2, 64, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
s, n = torch.ones(2, 2, 2), torch.zeros(2, dtype=torch.int32)
held = bind.cache(c, c.clone(), None, s, s.clone(), None)
for H in (3, -1):
    q = torch.zeros(2, abs(H), 1, 64, dtype=torch.bfloat16)
    try:
        if H > 0:
            bind.attn(held, q, None, n, None, True, None, None, 1.0, None, None, None)
        else:
            bind.append(held, None, q, q[:0], None, n, None)
    except ValueError as e:
        print(e)
try:                                     # an exception of torch's own, from one of its functions
    q = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16)
    bind.attn(held, q, None, n, None, True, None, None, 1.0, None, None, None)
except RuntimeError as e:
    print("torch:", len(str(e)) > 0)
libs = {line.split()[-1] for line in open("/proc/self/maps") if "libstdc++" in line}
print(len(libs))
"""
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert p.returncode == 0, (p.returncode, p.stderr[-2000:])
    assert p.stdout.splitlines() == ["3 query heads are not a multiple of the cache's 2",
                                     "k has shape (2, 1, 1, 64), expected (2, 2, 1, 64)",
                                     "torch: True", "1"]
