"""The word that says where a wait ran out, packed by a kernel and read on the
host: every kernel, barrier slot and warp that there is comes back."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_attention_backward_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "wait_site.h"
int main() {
  for (unsigned k = abw::kSiteKv; k < abw::kSiteEnd; ++k) {
    printf("%u %s\n", k, abw::site_kernel(k));
    for (unsigned slot = 0; slot < 128; ++slot)
      for (unsigned warp = 0; warp < 32; ++warp)
        for (unsigned block = 0; block < 65536; block += 257) {
          const abw::WaitSite s = abw::unpack_site(abw::pack_site({k, slot, warp, block}));
          if (s.kernel != k || s.slot != slot || s.warp != warp || s.block != block) return 1;
        }
  }
  return 0;
}
"""


def test_round_trip(tmp_path):
    src, exe = tmp_path / "site.cpp", tmp_path / "site"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], stdout=subprocess.PIPE, check=True).stdout.decode().splitlines()
    names = [line.split(" ", 1)[1] for line in out]
    assert len(names) == 7 and len(set(names)) == len(names) and "?" not in names


def test_every_kernel_of_the_linear_attention_has_a_site_of_its_own():
    lin = open(os.path.join(CSRC, "lin_attn.cu")).read()
    sites = re.findall(r"const LinWait lw\{[^}]*, (kSite\w+), ", lin)
    assert len(sites) == len(set(sites)) == 3
