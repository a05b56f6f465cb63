"""The check sites of the 8-bit kernels have numbers of their own too."""

from tests import test_sites


def test_sites_of_the_new_sources(monkeypatch):
    monkeypatch.setattr(test_sites, "LIBRARY", test_sites.LIBRARY + ("fa_serve8.cu", "fa_rotary.cu"))
    test_sites.test_every_site_has_a_number_of_its_own()
    test_sites.test_no_site_is_a_bare_number()
