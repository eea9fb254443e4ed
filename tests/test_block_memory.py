"""Memory order of the operators around the layer, on the CPU: which copies a block waits for before
it leaves early, and how operands are loaded."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "forward_moe_route_b200", "csrc")

# Every state in which a reader can give up: `rows` copies in all through `stages` slots, the wait
# for row `at` the first to run out, so rows up to at + stages were issued; those from `landed` on
# are on their way.  A barrier with c completed phases lets a wait for parity p pass if p != c & 1.
MODEL = r"""
#include <cstdio>
#include <vector>
#include "ring.h"

static long states = 0;

static bool covers(int stages, int rows, int at, int landed) {
  const int issued = at + stages < rows ? at + stages : rows;
  const int next = issued % stages;
  const uint32_t parity = (uint32_t)(issued / stages) & 1u;
  if (at < rows &&
      moe::ring_parity(next, at % stages, (uint32_t)(at / stages) & 1u) != parity) return false;
  std::vector<int> done(stages, 0), flying(stages, 0);
  for (int k = 0; k < issued; ++k) (k < landed ? done : flying)[k % stages] += 1;
  std::vector<int> calls(stages, 0);
  bool right = true;
  moe::ring_drain(next, parity, stages, [&](int s, uint32_t p) {
    ++calls[s];
    if (flying[s] > 1) right = false;
    if ((p != (done[s] & 1u)) != (flying[s] == 0)) right = false;       // waits exactly for these
    if (flying[s] && p == ((done[s] + 1) & 1u)) right = false;          // and passes once it landed
  });
  for (int s = 0; s < stages; ++s) right = right && calls[s] == 1;
  ++states;
  return right;
}

int main() {
  for (int stages = 1; stages <= 16; ++stages)
    for (int rows = 0; rows <= 4 * stages + 3; ++rows)
      for (int at = 0; at <= rows; ++at)
        for (int landed = at; landed <= rows && landed <= at + stages; ++landed)
          if (!covers(stages, rows, at, landed)) {
            printf("stages %d rows %d at %d landed %d\n", stages, rows, at, landed);
            return 1;
          }
  printf("%ld states\n", states);
  return 0;
}
"""


def test_a_reader_that_gives_up_waits_for_every_copy_on_its_way(tmp_path):
    (tmp_path / "model.cpp").write_text(MODEL)
    exe = tmp_path / "model"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "model.cpp"), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 10000


def test_every_kernel_with_a_ring_of_bulk_copies_drains_it():
    found = 0
    for name in ("norm.cuh", "adamw.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        # functions at namespace level: from a `template` or `__global__` line on
        parts = re.split(r"\n(?=template <|__global__|__device__|struct )", text)
        for part in parts:
            if part.startswith("struct ") or "struct SharedRow" in part:
                continue
            if re.search(r"bulk_load_1d\(|Row::copy\(", part):
                found += 1
                assert "bulk_drain(" in part, f"{name}: {part[:200]}"
    assert found == 3


def test_no_non_coherent_loads_behind_a_programmatic_launch():
    """The kernels of the operators around the layer may be launched while the kernel before them
    still writes their operands: ld.global.nc, which __ldg makes, is for data that stays as it is
    for a kernel's whole life."""
    for name in ("norm.cuh", "grouped.cuh", "grouped_few.cuh", "adamw.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert "grid_dep_sync();" in text, name
        assert not re.search(r"__ldg\(|ld\.global\.nc|__restrict__", text), name


def blocks_around(text, at):
    """The statements whose braces enclose position `at`."""
    heads, start = [], 0
    for i, c in enumerate(text[:at]):
        if c in "{};":
            if c == "{":
                heads.append(text[start:i])
            elif c == "}":
                heads.pop()
            start = i + 1
    return heads


def test_a_warp_gives_up_as_a_whole():
    """A wait that one lane gives up on while another sees its barrier complete would leave the
    second at the warp's next synchronising instruction for good: a wait whose outcome sends lanes
    different ways is one elected lane's, or the warp votes."""
    with open(os.path.join(CSRC, "grouped.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    one, warp = 0, 0
    for m in re.finditer(r"(?:!|= ?)mbar_wait(_warp)?\(", text):
        elected = any("elect_one()" in h for h in blocks_around(text, m.start()))
        assert elected != bool(m.group(1)), text[m.start():m.start() + 80]
        one += elected
        warp += not elected
    assert one >= 4 and warp >= 4
