"""Lanes of a wave that pass values through LDS: a wave barrier alone keeps the
instruction scheduler from moving accesses across it, but not the optimiser from giving
a lane back what it stored itself.  Each barrier of the operators' kernels stands
between two fences of the wavefront."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FENCED = re.compile(r'__builtin_amdgcn_fence\(__ATOMIC_RELEASE, "wavefront"\);\s*__builtin_amdgcn_wave_barrier\(\);\s*'
                    r'__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE, "wavefront"\);')


def test_wave_barriers_are_fenced():
    found = 0
    for path in sorted(glob.glob(os.path.join(ROOT, "tile_dependency_pipelined_amd", "csrc", "cp_ops*"))):
        text = open(path).read()
        barriers = len(re.findall(r"__builtin_amdgcn_wave_barrier\(\)", text))
        assert barriers == len(FENCED.findall(text)), os.path.basename(path)
        found += barriers
    assert found
