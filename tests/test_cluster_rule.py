"""Cluster sizes on several devices of one process (csrc/clusters.h), against a model of the runtime: a function's
attribute for clusters of more than 8 CTAs belongs to one device, and a launch of 16 without it fails."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_long_kbar_b200", "csrc")

MODEL = r"""
#include <cstdio>
#include "clusters.h"
struct Device { bool allowed, can_set; int room; };
// what a call on the device launches: the CTAs of its clusters, or -1 where the runtime refuses them
int launch(Device& d, int want) {
  const int n = sgqa::cluster_ctas(want, [&] { d.allowed = d.allowed || d.can_set; return d.can_set; }, [&] { return d.room; });
  return n <= 8 || (d.allowed && d.room > 0) ? n : -1;
}
int main() {
  Device a{false, true, 9}, b{false, true, 9}, small{false, true, 0}, old{false, false, 9};
  Device* order[] = {&small, &a, &b, &old, &b, &a, &small};
  for (Device* d : order) std::printf("%d %d %d ", launch(*d, 16), launch(*d, 8), launch(*d, 1));
  a = Device{false, true, 9};  // a new context on the same device
  std::printf("%d", launch(a, 16));
}
"""


def test_each_device_is_asked(tmp_path):
    src, exe = tmp_path / "m.cpp", tmp_path / "m"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [8, 8, 1, 16, 8, 1, 16, 8, 1, 8, 8, 1, 16, 8, 1, 16, 8, 1, 8, 8, 1, 16]


def test_no_launch_of_the_cache_keeps_what_a_device_answered():
    """No function-local static but the driver's entry point, which is one for the process."""
    for name in sorted(os.listdir(CSRC)):
        if name.startswith("cache8"):
            text = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
            kept = [x.strip() for x in re.findall(r"^\s+static (?!constexpr|__device__).*$", text, re.M)]
            assert kept in ([], ["static EncodeTiled fn = nullptr;"]), (name, kept)
