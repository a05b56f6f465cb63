"""The numbers in the status word's detail name one wait or check each."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_04_gb300", "csrc")
LIBRARY = ("common.cuh", "serve.cuh", "fa_fwd.cu", "fa_bwd.cu", "fa_serve.cu", "fa_cache.cu")


def _source(name):
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


def test_every_site_has_a_number_of_its_own():
    sites = {}
    for name in LIBRARY:
        for body in re.findall(r"enum\s*\{([^}]*)\}", _source(name)):
            value = -1
            for item in (x.strip() for x in body.split(",")):
                if not item.startswith("SITE_"):
                    break
                key, _, number = (x.strip() for x in item.partition("="))
                value = int(number) if number else value + 1
                assert key not in sites
                sites[key] = value
    assert len(sites) > 40
    taken = {}
    for key, value in sites.items():
        assert value not in taken, f"{key} and {taken[value]} are both {value}"
        assert not 100 <= value < 108, f"{key} is a number of fa_debug.h"
        taken[value] = key


def test_no_site_is_a_bare_number():
    for name in LIBRARY:
        bare = re.findall(r"record_(?:check|error)\([^;{]*,\s*\d+\)", _source(name))
        assert not bare, f"{name}: {bare}"
