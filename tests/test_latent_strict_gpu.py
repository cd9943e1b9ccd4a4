"""The latent attention's shape tests with a check that no NaN passes: every owned row is finite, and within the
tolerance (`off <= tol`, which is false for NaN, where test_latent_gpu's `off > tol` is false too)."""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from tests import test_latent_gpu as base

pytestmark = pytest.mark.gpu

TESTS = ["test_heads_and_tokens", "test_lengths", "test_trees", "test_wide_tables", "test_lengths_of_wide_tables",
         "test_trees_of_wide_tables", "test_rows_of_wide_tables_that_see_little", "test_codes_of_wide_tables_that_do_not_matter",
         "test_errors_of_wide_tables", "test_rows_that_see_little", "test_first_tiles_unseen", "test_sharp_and_flat",
         "test_growing_logits", "test_unseen_codes_do_not_matter", "test_extremes_of_q", "test_errors", "test_many_units",
         "test_many_sequences", "test_strides_and_outputs", "test_repeats_streams_and_graphs", "test_short_tables",
         "test_trees_in_a_graph", "test_appended_and_read"]


class Strict(base.Batch):
    def check(self, out, skip=()):
        rows = [t for b in range(len(self.lens)) if b not in skip for t in range(self.cu_list[b], self.cu_list[b + 1])]
        assert torch.isfinite(out[rows]).all()
        want, weight, flat, reach = self.want()
        tol = np.abs(want) * 2.0 ** -8 + weight * (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -16.4 * reach) + flat * 2.0 ** -16
        assert np.all(np.abs(base.f64(out) - want)[rows] <= tol[rows])
        outside = [t for t in range(self.total) if not self.cu_list[0] <= t < self.cu_list[-1]]
        assert np.all(base.f64(out)[outside] == 9.0)


def cases():
    for name in TESTS:
        marks = [m.args for m in getattr(getattr(base, name), "pytestmark", []) if m.name == "parametrize"]
        keys = [[k.strip() for k in names.split(",")] for names, _ in marks]
        for values in itertools.product(*(v for _, v in marks)):
            args = {}
            for ks, v in zip(keys, values):
                args.update(zip(ks, v if len(ks) > 1 else [v]))
            yield pytest.param(name, args, id=name + "".join(f"-{v}" for v in args.values()).replace(" ", ""))


@pytest.mark.parametrize("name,args", list(cases()))
def test_strict(name, args, monkeypatch):
    monkeypatch.setattr(base, "Batch", Strict)
    getattr(base, name)(**args)


def test_the_check_sees_a_nan():
    b = Strict([40], [2], 3)
    out = b.run()
    b.check(out)
    out[1, 2, 100] = float("nan")
    with pytest.raises(AssertionError):
        b.check(out)
