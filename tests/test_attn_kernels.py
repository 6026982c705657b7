"""Of linear attention's walks the library holds the kernels that some call reaches, and no others."""
import os
import re
import shutil
import subprocess

import pytest

from selective_state_space_85_amd import _lib

SINGLE, WHOLE, ANY = range(3)


def launches(dk, dv):
    """The widths of the walks of each launch: forward, and the gradients in one launch or two."""
    def kind(k, v):
        return (k > 64) + (k > 128), (v > 64) + (v > 128)

    yield [(dk, dv)]
    yield from ([[(dk, dv), (dv, dk)]] if kind(dk, dv) == kind(dv, dk) else [[(dk, dv)], [(dv, dk)]])


def reached():
    out = set()
    for dtype, chunk in ((0, 4), (1, 8)):  # elements of 16 bytes
        for dk in range(1, 257):
            for dv in range(1, 257):
                for jobs in launches(dk, dv):
                    padded = next(p for p in (64, 96, 128, 192, 256) if max(k for k, _ in jobs) <= p)
                    waves = 2 if jobs[0][1] <= 64 else 4
                    widths = [w for j in jobs for w in j]
                    reads = [ANY] if min(widths) >= chunk else [SINGLE]
                    if all(w % chunk == 0 for w in widths):
                        reads.append(WHOLE)
                    out.update((dtype, padded, waves, r, s) for r in reads for s in (0, 1))
    return out


@pytest.mark.skipif(shutil.which("nm") is None, reason="nm not available")
@pytest.mark.skipif("SS_SANITIZED_LIB" in os.environ, reason="this is the sanitized run")
def test_every_kernel_is_reached():
    if not os.path.exists(_lib.LIB_PATH):
        from selective_state_space_85_amd import build

        build.build()
    names = subprocess.run(["nm", _lib.LIB_PATH], check=True, capture_output=True, text=True).stdout
    held = {tuple(map(int, m)) for m in re.findall(r"lattn_kernelILi(\d)ELi(\d+)ELi(\d)ELNS0_6AccessE(\d)ELb(\d)", names)}
    assert held == reached(), held ^ reached()
