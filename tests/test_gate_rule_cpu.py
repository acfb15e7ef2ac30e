"""A routing rule is a value: it can be copied, compared, saved and handed to another process."""
import copy
import dataclasses
import pickle

import pytest

from sparse_moe_fine_gb300 import binding as B

RULE = B.Gate(score="sigmoid", n_group=8, topk_group=4, group_top=2, renorm=1, scale=2.5)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda g: pickle.loads(pickle.dumps(g)),
                                 lambda g: copy.deepcopy({"gate": [g]})["gate"][0], dataclasses.replace],
                         ids=["copy", "deepcopy", "pickle", "in_a_dict", "replace"])
@pytest.mark.parametrize("rule", [RULE, B.Gate()], ids=["sigmoid", "default"])
def test_copies_are_the_same_rule(how, rule):
    got = how(rule)
    assert got is not rule and got == rule and hash(got) == hash(rule)
    c = got._ref._obj                                         # what the library is handed is the copy's own
    assert c is got._c and c is not rule._c
    assert (c.score, c.n_group, c.topk_group, c.group_top, c.renorm, c.scale) == (
        B.SCORES[rule.score], rule.n_group, rule.topk_group, rule.group_top, rule.renorm, rule.scale)
