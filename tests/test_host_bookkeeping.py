"""Host-side bookkeeping of libcpa.so that needs no GPU.

The kernels' shared-memory limit and the static scratch's device address are
per-device facts: a process that drives several GPUs through one library
instance must set up each device, once.  The helper that remembers this
(``csrc/cpa_host.h``) is compiled here with the host C++ compiler alone and
driven with fake device indices and a fake set-up step.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "cascade_paged_attention_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "cpa_host.h"

int main() {
    cpa::PerDevice<int> pd;
    int calls[cpa::kMaxDevices] = {};
    int fail_next = 1;  // the first set-up of device 3 fails
    auto setup = [&](int dev) {
        return [&, dev](int& v) {
            ++calls[dev];
            if (dev == 3 && fail_next) { fail_next = 0; return 7; }
            v = 100 + dev;
            return 0;
        };
    };
    int out = -1;
    // device 0: set up once, remembered
    if (pd.run(0, -9, setup(0), &out) != 0 || out != 100) return 1;
    if (pd.run(0, -9, setup(0), &out) != 0 || out != 100 || calls[0] != 1) return 2;
    // device 1 is independent of device 0
    if (pd.run(1, -9, setup(1), &out) != 0 || out != 101 || calls[1] != 1) return 3;
    // a failed set-up is reported and retried on the next call
    if (pd.run(3, -9, setup(3), &out) != 7) return 4;
    if (pd.run(3, -9, setup(3), &out) != 0 || out != 103 || calls[3] != 2) return 5;
    // device indices outside the table
    if (pd.run(-1, -9, setup(0)) != -9 || pd.run(cpa::kMaxDevices, -9, setup(0)) != -9) return 6;
    // many threads racing on a new device run its set-up exactly once
    std::vector<std::thread> ts;
    for (int i = 0; i < 16; ++i)
        ts.emplace_back([&] { int o = 0; pd.run(5, -9, setup(5), &o); });
    for (auto& t : ts) t.join();
    if (calls[5] != 1) return 7;
    std::printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_per_device_setup_runs_once_per_device(tmp_path):
    src = tmp_path / "harness.cpp"
    exe = tmp_path / "harness"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)


JOINS = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include "cpa_types.h"

int main() {
    // whatever an entry holds: what passes names a unit of the call and parts that exist
    std::srand(7);
    auto word = [] {
        const uint32_t r = (uint32_t)std::rand() * 2654435761u;
        switch (r % 5) {
            case 0: return (int)r;
            case 1: return (int)(r >> 8) % 160 - 4;
            case 2: return (int)0xA5A5A5A5u;
            case 3: return 0x7fffffff;
            default: return (int)(r >> 16) % 9 - 1;
        }
    };
    long long passed = 0;
    for (int i = 0; i < 3000000; ++i) {
        const int B = 1 + std::abs(word() % 200), n_pairs = 1 + std::abs(word() % 7), n_grp = i & 1 ? 152 : 76;
        const int b = word(), pair = word(), parts = word(), group = word();
        if (!cpa::join_in_range(b, pair, parts, group, B, n_pairs, n_grp)) continue;
        ++passed;
        if (b < 0 || b >= B || pair < 0 || pair >= n_pairs || parts < 2) return 1;
        if (group < 0 || (long long)group + parts > n_grp) return 2;
    }
    if (passed < 100) return 3;
    // what a call writes passes
    if (!cpa::join_in_range(0, 0, 152, 0, 1, 1, 152) || !cpa::join_in_range(63, 1, 2, 150, 64, 2, 152)) return 4;
    // units that are whole, or begin nowhere, are nobody's to join
    if (cpa::join_in_range(0, 0, 1, 0, 1, 1, 152) || cpa::join_in_range(-1, 0, 0, 0, 1, 1, 152)) return 5;
    std::printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_a_join_stays_in_bounds_whatever_its_entry_holds(tmp_path):
    src, exe = tmp_path / "joins.cpp", tmp_path / "joins"
    src.write_text(JOINS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
    # and the join whose entries a block may have left unwritten looks at nothing before it asks
    with open(os.path.join(CSRC, "cpa_latent.cu")) as f:
        text = f.read()
    join = text[text.index("latent_join_kernel(const"):]
    assert join.index("join_in_range(d.x, d.y, d.z, d.w") < join.index("const Rows r(p, d.y")
